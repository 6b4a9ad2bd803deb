// Attention of drafted tokens over a paged Q8_0 cache (epq_attention_tree).
//
//   s_ij = scale q_i . k_j,  o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// over the committed positions and the drafted tokens that token i's mask
// names.  The rows of one (sequence, key/value head) are its tokens times its
// `group` query heads (row r: token r / group, head r % group); a row tile is
// 16 WM of them.
//
// One pass over the positions in tiles of 64, a running maximum per row, and
// both products on the tensor cores (mma.sync m16n8k16, 16-bit operands, float32
// sums) without giving up float32 accuracy:
//   scores   the int8 codes of a key are exact in fp16; a query row is scaled
//            by a power of two and split into two fp16 parts (2^-22 of the
//            entry, or 2^-38 of the row's largest); the sum of one 32-element
//            block is multiplied by that key's block factor in float32.
//   values   the codes are again the operand; the factor of (position, block)
//            goes to the other side: warp b owns the 32 columns of block b and
//            multiplies the weights by that block's factors.  A weight is kept
//            as two fp16 parts, so a product is three half2 operations: its
//            rounded value, what the rounding lost (exact), plus the second
//            part's product: 2^-22 of it, or 2^-34 of one at the reference with
//            the largest factor that block b has in the tile (a power of two
//            brings that factor into [1, 2)).
//            That floor would show where every larger weight meets a code 0, so
//            a tile with a weight below 2^-14 (times the factor's share of the
//            tile's largest) in a row that has not had 12 larger ones takes
//            float32 products in three bf16 parts, which lose nothing; so does
//            a warp whose block has factors more than 2^6 apart.
// The weights of a row are relative to its maximum at some earlier tile (the
// reference), which moves, and the sums with it, only when a weight passes 2^6:
// so the warps need not agree on a maximum before they form weights, and one
// barrier per tile is enough.
// Work: the tiles of all (sequence, head, row tile) items in a row, cut into
// equal shares, one per CTA.  An item counts kExtra tiles more than it has:
// beginning it, and its last tile with the new rows, take that long.  A CTA's
// part of an item that it does not hold whole goes to the workspace (maximum,
// sum, unnormalised output), and a second launch joins the parts in the order
// of their positions.
// Warp 0 streams the rows of a tile (contiguous within a page) with bulk
// copies into a ring of three stages, two tiles ahead; the warps of a row
// group compute the scores of 64 / (D/32) positions each, exchange the weights
// through shared memory (one barrier per tile) and accumulate 32 columns each.
// The new rows are quantized into their tile by the CTAs that read it (the
// one of row tile 0 also stores them in the cache).
// Measured with 32 query and 8 key/value heads of 128 (both launches, from a
// graph): 64 tokens over 8193 positions 107 us, four sequences of 8 tokens over
// 32 k positions 174 us (280 MB of cache, 1.6 TB/s), 8 tokens over 1024
// positions 18 us, one token over 37 positions 10 us; heads of 256: 196, 344,
// 19 and 10 us.  The long ones are bound
// by instructions between the products, 0.52 issued per cycle of a scheduler
// with 4 warps each (the MMA pipe is 31 % busy): a warp spends ~870 on a tile
// of 16 rows, 64 of them MMAs.  Short ones are one chain of tile, parts and
// join.  32 rows per warp take a third fewer instructions but leave half the
// warps: 113, 167, 20 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "pages.cuh"

namespace epq {
namespace {

constexpr int kTile = 64;  // positions of a tile
constexpr int kStages = 3;
constexpr int kMaxGroupTree = 16;
constexpr int kMaxCtas = 512;
constexpr int kJoinThreads = 128;
constexpr int kExtra = 2;            // tiles' worth of work that an item has besides its tiles
struct TreeParams {
  PagesView v;
  const float *q, *k_new, *v_new;
  const uint64_t *mask;
  const int32_t *n_tok;
  int64_t q_ld, q_seq_ld, kv_ld, kv_seq_ld;
  int layer, n_heads, group, ntok;
  float scale;
  float *out;
  long long *before;  // workspace: tiles of the sequences before each, then their total
  float *parts;       // workspace: [2 per CTA][rows][D + 4]
  unsigned *err;
};

__device__ __forceinline__ int tree_size(const TreeParams &p, int s) {
  return p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok;
}

// Tiles of one row tile of a sequence with n tokens; what
// the item counts in the shares is kExtra more.
__device__ __forceinline__ int sequence_tiles(int len, int n) { return n ? (len + n + kTile - 1) / kTile : 0; }

__device__ __forceinline__ uint64_t token_mask(const TreeParams &p, int s, int i, int n) {
  const uint64_t m = p.mask ? p.mask[s * p.ntok + i] : ~0ull >> (63 - i);
  return n >= 64 ? m : m & ((1ull << n) - 1);
}

// Shares of `total` tiles: CTA c holds [c share + min(c, rest), ...).
struct Shares {
  long long share, rest;
  __device__ Shares(long long total, int ctas) : share(total / ctas), rest(total % ctas) {}
  __device__ long long begin(long long c) const { return c * share + (c < rest ? c : rest); }
  __device__ int holder(long long x) const {
    const long long cut = rest * (share + 1);
    return static_cast<int>(x < cut ? x / (share + 1) : rest + (x - cut) / share);
  }
};

constexpr float kUp = 9.0f;           // log2 of a weight at its row's reference as it is held
constexpr float kPast = 32768.0f;     // largest weight as it is held: 2^6 at the reference
constexpr float kWeighty = 0.03125f;  // a weight that counts, as it is held: 2^-14 at the reference
constexpr float kWeightyMin = 12.0f;  // of them, among a warp's positions
constexpr float kApart = 0.015625f;   // 2^-6: down to this share of its tile's largest a factor takes fp16 parts

// What a work item is: row tile rt of head h of sequence s.
struct Item {
  int s, h, rt, tiles, len, n;
};

// The work of a launch, in shared memory: lengths and tokens of the sequences,
// the tiles (kExtra more per item) before each of them, and the CTA's share.
struct Work {
  long long before[kMaxSeq + 1], begin, end;
  int2 seq[kMaxSeq];
};

// Filled by warp 0; ends with a CTA barrier.
template <int kRows>
__device__ __forceinline__ void find_work(const TreeParams &p, Work &wk) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    long long run = 0;
    for (int s0 = 0; s0 < p.v.n_seq; s0 += 32) {
      long long x = 0;
      if (s0 + lane < p.v.n_seq) {
        const int n = tree_size(p, s0 + lane), len = seq_length(p.v, s0 + lane);
        wk.seq[s0 + lane] = make_int2(len, n);
        const int tiles = sequence_tiles(len, n);
        x = static_cast<long long>(tiles ? tiles + kExtra : 0) * ((n * p.group + kRows - 1) / kRows) * p.v.n_kv;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (s0 + lane < p.v.n_seq) wk.before[s0 + lane + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      wk.before[0] = 0;
      const int ctas = static_cast<int>(run < gridDim.x ? run : gridDim.x);
      wk.begin = wk.end = 0;
      if (blockIdx.x < ctas) {
        const Shares sh(run, ctas);
        wk.begin = sh.begin(blockIdx.x);
        wk.end = sh.begin(blockIdx.x + 1);
      }
    }
  }
  __syncthreads();
  if (blockIdx.x == 0)  // for the join
    for (int s = threadIdx.x; s <= p.v.n_seq; s += blockDim.x) p.before[s] = wk.before[s];
}

// The item that holds unit x of the work, and the unit's place in it (from
// it.tiles on: none of its tiles).
template <int kRows>
__device__ __forceinline__ int find_item(const TreeParams &p, const Work &wk, long long x, Item &it) {
  int lo = 0, hi = p.v.n_seq - 1;
  while (lo < hi) {  // the last sequence with before[s] <= x (empty ones are passed over)
    const int mid = (lo + hi + 1) / 2;
    if (wk.before[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  it.s = lo;
  it.len = wk.seq[lo].x;
  it.n = wk.seq[lo].y;
  it.tiles = sequence_tiles(it.len, it.n);
  const int nrt = (it.n * p.group + kRows - 1) / kRows;
  const long long rel = x - wk.before[lo];
  const int units = it.tiles + kExtra;
  int k, tile;
  if (rel >> 31) {
    k = static_cast<int>(rel / units);
    tile = static_cast<int>(rel % units);
  } else {
    k = static_cast<int>(rel) / units;
    tile = static_cast<int>(rel) - k * units;
  }
  it.h = k / nrt;
  it.rt = k - it.h * nrt;
  return tile;
}

// The outputs of tokens beyond a sequence's tree are 0.
__device__ __forceinline__ void clear_unused(const TreeParams &p, const Work &wk) {
  if (!p.n_tok) return;
  const int width = p.n_heads * p.v.D;
  for (int r = blockIdx.x; r < p.v.n_seq * p.ntok; r += gridDim.x) {
    if (r % p.ntok < wk.seq[r / p.ntok].y) continue;
    float4 *o = reinterpret_cast<float4 *>(p.out + static_cast<int64_t>(r) * width);
    for (int i = threadIdx.x; i < width / 4; i += blockDim.x) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// Where row `row` of head h of sequence s goes.
__device__ __forceinline__ float *out_row(const TreeParams &p, int s, int h, int row) {
  return p.out + (static_cast<int64_t>(s) * p.ntok + row / p.group) * p.n_heads * p.v.D +
         (h * p.group + row % p.group) * p.v.D;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// Two codes as fp16: a byte u = code + 128 under the byte 0x64 is the half
// 1024 + u.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t x, uint32_t sel) {
  return as_bits(__hsub2(as_half2(__byte_perm(x, 0x64646464u, sel)), __half2half2(__ushort_as_half(0x6480))));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// x, y -> fp16 parts: first = rounded, second = the rest rounded.
__device__ __forceinline__ void split_half2(float x, float y, uint32_t &first, uint32_t &rest) {
  first = pack_half2(x, y);
  const float2 f = __half22float2(as_half2(first));
  rest = pack_half2(x - f.x, y - f.y);
}

__device__ __forceinline__ float f16_at(const uint8_t *p) {
  return __half2float(__ushort_as_half(*reinterpret_cast<const unsigned short *>(p)));
}

__device__ __forceinline__ float half_value(uint32_t bits) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Joins the parts of the items that more than one CTA holds: one warp per
// (item, row), the parts in the order of their positions.
template <int kD, int kRows>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ TreeParams p, int grid) {
  constexpr long long kPart = kRows * (kD + 4);
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.y, lane = threadIdx.x & 31;
  const int x = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);  // (head, row of the head)
  const int rows = p.ntok * p.group, h = x / rows, row = x - h * rows;
  const long long first = p.before[s], total = p.before[p.v.n_seq];
  const int n = tree_size(p, s);
  const int tiles = sequence_tiles(seq_length(p.v, s), n);
  if (h >= p.v.n_kv || row >= n * p.group) return;
  const int nrt = (n * p.group + kRows - 1) / kRows;
  const Shares sh(total, static_cast<int>(grid < total ? grid : total));
  const long long i0 = first + static_cast<long long>(h * nrt + row / kRows) * (tiles + kExtra);
  const int c0 = sh.holder(i0), c1 = sh.holder(i0 + tiles - 1);
  if (c0 == c1) return;  // one CTA held it whole and wrote it
  // only the first of the item's CTAs can have begun before it
  const float *rest = p.parts + (row % kRows) * (kD + 4);
  const float *head = rest + (sh.begin(c0) >= i0 ? 0 : kPart);
  auto part = [&](int c) { return (c == c0 ? head : rest) + 2 * kPart * c; };
  float top = -INFINITY, den = 0.0f;
  float4 y[kD / 128] = {};
  for (int b = c0; b <= c1; b += 32) {  // 32 parts at a time: a lane holds the maximum and sum of one
    const int m = min(32, c1 - b + 1);
    const float2 ml = lane < m ? *reinterpret_cast<const float2 *>(part(b + lane) + kD) : make_float2(-INFINITY, 0.0f);
    const float up = fmaxf(top, warp_max_all(ml.x));
    const float ref = up == -INFINITY ? 0.0f : up;
    const float keep = exp2f(top - ref), f = exp2f(ml.x - ref);  // 0 for a part that saw nothing
    top = up;
    den = fmaf(den, keep, warp_sum_xor<32>(f * ml.y));
#pragma unroll
    for (int e = 0; e < kD / 128; ++e) y[e].x *= keep, y[e].y *= keep, y[e].z *= keep, y[e].w *= keep;
#pragma unroll 8
    for (int c = 0; c < m; ++c) {
      const float fc = __shfl_sync(0xffffffffu, f, c);
      const float4 *src = reinterpret_cast<const float4 *>(part(b + c)) + lane;
#pragma unroll
      for (int e = 0; e < kD / 128; ++e) {
        const float4 a = src[32 * e];
        y[e].x = fmaf(fc, a.x, y[e].x);
        y[e].y = fmaf(fc, a.y, y[e].y);
        y[e].z = fmaf(fc, a.z, y[e].z);
        y[e].w = fmaf(fc, a.w, y[e].w);
      }
    }
  }
  float *out = p.out + (static_cast<int64_t>(s) * p.ntok + row / p.group) * p.n_heads * kD +
               (h * p.group + row % p.group) * kD;
#pragma unroll
  for (int e = 0; e < kD / 128; ++e)
    *reinterpret_cast<float4 *>(out + 128 * e + 4 * lane) =
        den != 0.0f ? make_float4(y[e].x / den, y[e].y / den, y[e].z / den, y[e].w / den) : make_float4(0.f, 0.f, 0.f, 0.f);
}

template <int kD, int kRows>
cudaError_t launch_join(const TreeParams &p, int grid, cudaStream_t s) {
  const int rows = p.v.n_kv * p.ntok * p.group, per = kJoinThreads / 32;
  return launch_pdl(join_kernel<kD, kRows>, dim3((rows + per - 1) / per, p.v.n_seq), dim3(kJoinThreads), 0, s, p, grid);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Two codes (bytes c of x picked by sel) as bf16: under the byte 0x43 the low
// seven bits are 128 + (c & 127), and 0x4300 | (c & 128) is 128, or 256 for a
// negative code; their difference is c, exactly.
__device__ __forceinline__ uint32_t codes_to_bf162(uint32_t x, uint32_t sel) {
  const uint32_t h = __byte_perm(x, 0x43434343u, sel);
  const uint32_t m = h & 0xff7fff7fu, n = h & 0xff80ff80u;
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&m), *reinterpret_cast<const __nv_bfloat162 *>(&n));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// x, y as the sum of three bf16 parts: 8 bits of the significand each.
__device__ __forceinline__ void split_bf162(float x, float y, uint32_t &p1, uint32_t &p2, uint32_t &p3) {
  p1 = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
  p2 = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
  p3 = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}

template <int NB, int WM>
struct Plan {
  static constexpr int kD = 32 * NB;
  static constexpr int kRow = kD + kD / 16;
  static constexpr int kRows = 16 * WM;
  static constexpr int kWarps = NB * WM;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kKeys = kTile / NB;  // positions whose scores a warp computes
  static constexpr int kNT = kKeys / 8;
  static constexpr uint32_t kStageBytes = 2u * kTile * kRow;
  static constexpr int kPart = kRows * (kD + 4);  // floats of a part
  // shared memory (bytes)
  static constexpr uint32_t oStage = 0;
  static constexpr uint32_t oQ = oStage + kStages * kStageBytes;    // query fragments, two parts
  static constexpr uint32_t oW = oQ + 2u * 2u * kRows * kD;         // [2][rows][64] weights
  static constexpr uint32_t oMax = oW + 2u * 4u * kRows * kTile;    // [NB][rows] maxima
  static constexpr uint32_t oSum = oMax + 4u * NB * kRows;          // [NB][rows]
  static constexpr uint32_t oMask = oSum + 4u * NB * kRows;         // [rows] mask words
  static constexpr uint32_t oScale = oMask + 8u * kRows;            // [rows] score factors (log2 units)
  static constexpr uint32_t oWork = oScale + 4u * kRows;            // Work
  static constexpr uint32_t oBar = oWork + sizeof(Work);            // full
  static constexpr uint32_t oTell = oBar + 8u * (kStages + 1);      // [2][warps] see `tell`
  static constexpr uint32_t oMiss = oTell + 2u * 8u * kWarps;       // [stages] missing pieces
  static constexpr uint32_t kSmem = oMiss + 4u * kStages + 4u;
};

template <int NB, int WM>
__global__ void __launch_bounds__(Plan<NB, WM>::kThreads, NB == 4 ? (WM == 1 ? 3 : 2) : 1)
    tree_kernel(const __grid_constant__ TreeParams p) {
  using L = Plan<NB, WM>;
  constexpr int kRows = L::kRows, kD = L::kD, kRow = L::kRow, kNT = L::kNT, kOwn = 2 * kNT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp / NB, wb = warp % NB;  // rows 16 wm ..., positions wb kKeys ..., columns 32 wb ...
  const int g = lane >> 2, t = lane & 3;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::oBar);
  Work &wk = *reinterpret_cast<Work *>(smem + L::oWork);
  unsigned *miss = reinterpret_cast<unsigned *>(smem + L::oMiss);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  find_work<kRows>(p, wk);
  clear_unused(p, wk);
  const long long begin = wk.begin, end = wk.end;
  if (begin == end) return;
  auto find = [&](long long x, Item &it) { return find_item<kRows>(p, wk, x, it); };
  const int piece_rows = min(p.v.P, kTile);

  // ---------------------------------------------------------------- loads
  // Warp 0 copies a tile's committed rows: lane 2 piece + plane takes the rows
  // of one page (at most four of them in a tile).  The page ids are read a
  // tile earlier than they are needed.
  Item load_it = {};
  int load_tile = 0, load_rows = 0, load_page = 0;
  long long load_x = begin;
  uint32_t load_k = 0;
  auto look_ahead = [&]() {
    // to the next tile that there is (none of what an item counts beyond them)
    while (load_x < end && (load_x == begin || load_tile >= load_it.tiles)) {
      if (load_x != begin) load_x += load_it.tiles + kExtra - load_tile;
      if (load_x >= end) break;
      load_tile = find(load_x, load_it);
      if (load_tile < load_it.tiles) break;
      load_x += load_it.tiles + kExtra - load_tile;
      load_tile = load_it.tiles + kExtra;  // the next turn finds the item that begins here
    }
    if (load_x >= end) return;
    const int pos = load_tile * kTile + (lane >> 1) * piece_rows;
    load_rows = (lane >> 1) < kTile / piece_rows ? min(max(load_it.len - pos, 0), piece_rows) : 0;
    load_page = load_rows > 0 ? p.v.table[static_cast<int64_t>(load_it.s) * p.v.max_pages + pos / p.v.P] : 0;
  };
  auto load = [&]() {
    if (load_x >= end) return;
    const int st = load_k % kStages, piece = lane >> 1, c = lane & 1;
    const bool page_ok = load_page >= 0 && load_page < p.v.n_pages;
    const uint32_t bytes = load_rows > 0 && page_ok ? (static_cast<uint32_t>(load_rows) * kRow) & ~15u : 0u;
    const unsigned lost = __ballot_sync(0xffffffffu, !page_ok);
    if (lost && lane == 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(load_it.s));
    const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
    if (lane == 0) {
      miss[st] = lost;
      if (all) mbar_arrive_expect_tx(&full[st], all);
      else mbar_arrive(&full[st]);
    }
    __syncwarp();
    if (bytes)
      bulk_g2s(smem + L::oStage + st * L::kStageBytes + (c * kTile + piece * piece_rows) * kRow,
               page_row(p.v, p.layer, load_page, load_it.h, c, (load_tile * kTile + piece * piece_rows) % p.v.P), bytes,
               &full[st]);
    ++load_tile;
    ++load_x;
    ++load_k;
  };
  if (warp == 0) {
    look_ahead();
    load();
    look_ahead();
    load();
    look_ahead();
  }

  uint64_t *row_mask = reinterpret_cast<uint64_t *>(smem + L::oMask);
  float *row_scale = reinterpret_cast<float *>(smem + L::oScale);
  float *sums = reinterpret_cast<float *>(smem + L::oSum);
  bool ok = true;
  uint32_t k = 0;
  for (long long x = begin; x < end;) {
    Item it;
    const int first = find(x, it);
    const int last = static_cast<int>(min(static_cast<long long>(it.tiles), first + (end - x)));
    const long long x0 = x;
    x += it.tiles + kExtra - first;
    if (first >= it.tiles) continue;
    const int n_rows = min(kRows, it.n * p.group - it.rt * kRows);

    // -------------------------------------------------------------- queries
    // A warp takes rows: scaled by a power of two so that the largest entry
    // is in [2^13, 2^14), split, stored as MMA A fragments (element 16 ks +
    // 4 t + e: lane t of the row, register e / 2).
    {
      constexpr int kPer = 16 / NB;  // rows of a warp
      float4 q[kPer][NB / 4];
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int r = warp + L::kWarps * u, row = it.rt * kRows + r, i = row / p.group;
#pragma unroll
        for (int c = 0; c < NB / 4; ++c)
          q[u][c] = r < n_rows ? *reinterpret_cast<const float4 *>(p.q + it.s * p.q_seq_ld + i * p.q_ld +
                                                                   (it.h * p.group + row % p.group) * kD + 128 * c +
                                                                   4 * lane)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane == 0) row_mask[r] = r < n_rows ? token_mask(p, it.s, i, it.n) : 0;
      }
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int r = warp + L::kWarps * u;
        float a = 0.0f;
#pragma unroll
        for (int c = 0; c < NB / 4; ++c)
          a = fmaxf(fmaxf(a, fmaxf(fabsf(q[u][c].x), fabsf(q[u][c].y))), fmaxf(fabsf(q[u][c].z), fabsf(q[u][c].w)));
        a = warp_absmax(a);
        const int e = min(max(static_cast<int>(__float_as_uint(a) >> 23) - 127, -100), 127);
        const float up = exp2i(13 - e);
        if (lane == 0) row_scale[r] = p.scale * 1.4426950408889634f * exp2i(e - 13);
#pragma unroll
        for (int c = 0; c < NB / 4; ++c) {
          uint32_t h0, h1, l0, l1;
          split_half2(q[u][c].x * up, q[u][c].y * up, h0, l0);
          split_half2(q[u][c].z * up, q[u][c].w * up, h1, l1);
          // float4 index 32 c + lane = 4 (16-element step) + t
          uint32_t *f = reinterpret_cast<uint32_t *>(smem + L::oQ) +
                        (((r >> 4) * (2 * NB) + 8 * c + g) * 2 * 32 + (r & 7) * 4 + t) * 4 + ((r >> 3) & 1);
          f[0] = h0;
          f[2] = h1;
          f[128] = l0;
          f[130] = l1;
        }
      }
    }
    __syncthreads();

    float o[4][4] = {}, s[2][kOwn];  // s: scores, then weights, of rows g, g + 8 at the lane's positions
    float ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {}, weighty[2] = {};
    const float c_row[2] = {row_scale[16 * wm + g], row_scale[16 * wm + 8 + g]};
    float unit = 1.0f;  // power of two on the value factors of the warp's columns: a tile's largest comes into [1, 2)
    uint32_t largest = 0, smallest = 0;  // of these factors (fp16) in the tile

    // Scores of tile `tile` (pipeline step kk) into s.
    auto scores = [&](int tile, uint32_t kk) {
      const int st = kk % kStages;
      uint8_t *kt = smem + L::oStage + st * L::kStageBytes, *vt = kt + kTile * kRow;
      const int t0 = tile * kTile;
      bool special = t0 + kTile > it.len;
      if (special) {
        // While the committed rows are on their way (none of what is written
        // here is in their copies): the factors of rows that hold nothing are 0,
        for (int i = tid; i < 2 * kTile; i += L::kThreads) {
          const int r = i >> 1, pos = t0 + r;
          uint8_t *dst = (i & 1 ? vt : kt) + r * kRow;
          if (pos >= it.len + it.n) {
#pragma unroll
            for (int b = 0; b < NB / 4; ++b) reinterpret_cast<uint2 *>(dst)[b] = make_uint2(0, 0);
          } else if (pos == it.len - 1 && ((r % piece_rows + 1) * kRow & 8)) {
            // the end of an odd number of rows (a bulk copy moves 16 bytes),
            const int page = seq_page(p.v, it.s, pos / p.v.P);
            if (page >= 0)
              *reinterpret_cast<uint2 *>(dst + kRow - 8) =
                  *reinterpret_cast<const uint2 *>(page_row(p.v, p.layer, page, it.h, i & 1, pos % p.v.P) + kRow - 8);
          }
        }
        // and the new rows
        const int r0 = max(it.len - t0, 0), r1 = min(it.len + it.n - t0, kTile);
        constexpr int kBatch = NB == 4 ? 4 : 2;  // row planes of a warp whose loads are in flight together
        for (int rr0 = 2 * r0 + warp; rr0 < 2 * r1; rr0 += kBatch * L::kWarps) {
          float4 x[kBatch][NB / 4];
          int page[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int rr = min(rr0 + u * L::kWarps, 2 * r1 - 1), pos = t0 + (rr >> 1);
            const float *src = (rr & 1 ? p.v_new : p.k_new) + it.s * p.kv_seq_ld + (pos - it.len) * p.kv_ld + it.h * kD;
#pragma unroll
            for (int b = 0; b < NB / 4; ++b) x[u][b] = *reinterpret_cast<const float4 *>(src + 128 * b + 4 * lane);
            page[u] = it.rt == 0 ? seq_page(p.v, it.s, pos / p.v.P) : -1;
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int rr = rr0 + u * L::kWarps;
            if (rr >= 2 * r1) break;
            const int r = rr >> 1, c = rr & 1, pos = t0 + r;
            uint8_t *dst = (c ? vt : kt) + r * kRow, *row = nullptr;
            if (page[u] >= 0) row = page_row(p.v, p.layer, page[u], it.h, c, pos % p.v.P);
            else if (it.rt == 0 && lane == 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(it.s));
#pragma unroll
            for (int b = 0; b < NB / 4; ++b) {
              __half d;
              const uint32_t word = quantize4(x[u][b], &d);
              const int at = kD / 16 + 128 * b + 4 * lane, fat = 2 * (4 * b + (lane >> 3));
              *reinterpret_cast<uint32_t *>(dst + at) = word;
              if ((lane & 7) == 0) *reinterpret_cast<uint16_t *>(dst + fat) = __half_as_ushort(d);
              if (row) {
                *reinterpret_cast<uint32_t *>(row + at) = word;
                if ((lane & 7) == 0) *reinterpret_cast<uint16_t *>(row + fat) = __half_as_ushort(d);
              }
            }
          }
        }
      }
      if (ok) ok = mbar_wait_poll(&full[st], (kk / kStages) & 1, p.err, DEVERR_FULL_WAIT, kk);
      const unsigned lost = miss[st];
      if (lost) {  // rows of a missing page: no factors, and masked below
        special = true;
        for (int i = tid; i < 2 * kTile; i += L::kThreads) {
          const int r = i >> 1;
          if (t0 + r < it.len && lost >> (2 * (r / piece_rows)) & 1)
#pragma unroll
            for (int b = 0; b < NB / 4; ++b)
              reinterpret_cast<uint2 *>((i & 1 ? vt : kt) + r * kRow)[b] = make_uint2(0, 0);
        }
      }
      if (special) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
      }
      const uint8_t *kw = kt + wb * L::kKeys * kRow;
      uint2 four[kOwn];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) s[0][j] = s[1][j] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t kb[kNT][4];
#pragma unroll
        for (int j = 0; j < kNT; ++j) {  // column n of MMA tile j: position kNT n + j
          const uint8_t *r = kw + (kNT * g + j) * kRow + kD / 16 + 32 * b + 4 * t;
          const uint32_t w0 = *reinterpret_cast<const uint32_t *>(r) ^ 0x80808080u;
          const uint32_t w1 = *reinterpret_cast<const uint32_t *>(r + 16) ^ 0x80808080u;
          kb[j][0] = codes_to_half2(w0, 0x4140);
          kb[j][1] = codes_to_half2(w0, 0x4342);
          kb[j][2] = codes_to_half2(w1, 0x4140);
          kb[j][3] = codes_to_half2(w1, 0x4342);
        }
        float acc[kNT][4] = {};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const uint4 *f = reinterpret_cast<const uint4 *>(smem + L::oQ) + (wm * (2 * NB) + 2 * b + ks) * 64 + lane;
          const uint4 hi = f[0], lo = f[32];
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            mma_f16(acc[j], hi, kb[j][2 * ks], kb[j][2 * ks + 1]);
            mma_f16(acc[j], lo, kb[j][2 * ks], kb[j][2 * ks + 1]);
          }
        }
        float d[kOwn];  // factors of the lane's positions kOwn t ..., read four blocks at a time
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          if (b % 4 == 0) four[j] = *reinterpret_cast<const uint2 *>(kw + (kOwn * t + j) * kRow + 2 * b);
          const float2 two = __half22float2(as_half2(b & 2 ? four[j].y : four[j].x));
          d[j] = b & 1 ? two.y : two.x;
        }
#pragma unroll
        for (int j = 0; j < kNT; ++j) {
          s[0][j] = fmaf(d[j], acc[j][0], s[0][j]);
          s[0][kNT + j] = fmaf(d[kNT + j], acc[j][1], s[0][kNT + j]);
          s[1][j] = fmaf(d[j], acc[j][2], s[1][j]);
          s[1][kNT + j] = fmaf(d[kNT + j], acc[j][3], s[1][kNT + j]);
        }
      }
      // the range of the value factors that the warp's columns have in the tile
      // (a factor of 0 does not count)
      {
        const uint8_t *r = vt + lane * kRow + 2 * wb;
        uint32_t x = *reinterpret_cast<const unsigned short *>(r) & 0x7fffu;
        uint32_t y = *reinterpret_cast<const unsigned short *>(r + 32 * kRow) & 0x7fffu;
        if (special) {  // not finite: not in the products
          x = x < 0x7c00u ? x : 0u;
          y = y < 0x7c00u ? y : 0u;
        }
        largest = __reduce_max_sync(0xffffffffu, max(x, y));
        smallest = __reduce_min_sync(0xffffffffu, min(x ? x : 0x7c00u, y ? y : 0x7c00u));
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int j = 0; j < kOwn; ++j) s[b][j] *= c_row[b];
      if (special) {
        // A value factor that is not finite counts as 0 in the products; a row
        // that sees it, or a score that is not finite, becomes NaN here, which
        // moves no reference: the other rows' results stay as they are.
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const int r = wb * L::kKeys + kOwn * t + j, i = t0 + r - it.len;
          float bad = 0.0f;
#pragma unroll
          for (int b = 0; b < NB; ++b) bad += 0.0f * f16_at(vt + r * kRow + 2 * b);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint64_t may = row_mask[16 * wm + 8 * b + g];
            const bool see = i < 0 ? !(lost >> (2 * (r / piece_rows)) & 1) : i < 64 && (may >> i & 1);
            s[b][j] = see ? s[b][j] + fmaf(s[b][j], 0.0f, bad) : -INFINITY;
          }
        }
      }
    };

    // A turn: scores and weights of a tile, the barrier, its values; a turn whose
    // weights pass the reference too far begins again with a new one.
    bool fresh = true;
#pragma unroll 1
    for (int tile = first; tile < last;) {
      const int st = k % kStages;
      scores(tile, k);
      if (fresh) {  // new references
        float *mx = reinterpret_cast<float *>(smem + L::oMax) + 16 * wm + g;
        float m[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          m[b] = -INFINITY;
#pragma unroll
          for (int j = 0; j < kOwn; ++j) m[b] = fmaxf(m[b], s[b][j]);
          m[b] = fmaxf(m[b], __shfl_xor_sync(0xffffffffu, m[b], 1));
          m[b] = fmaxf(m[b], __shfl_xor_sync(0xffffffffu, m[b], 2));
          if (t == 0) mx[wb * kRows + 8 * b] = m[b];
        }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float top = ref[b];
#pragma unroll
          for (int c = 0; c < NB; ++c) top = fmaxf(top, mx[c * kRows + 8 * b]);
          const float keep = ref[b] == top ? 1.0f : exp2_approx(ref[b] - top);
          ref[b] = top;
          l_run[b] *= keep;
          weighty[b] *= keep;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[j][2 * b] *= keep;
            o[j][2 * b + 1] *= keep;
          }
        }
      }
      // ------------------------------------------------------------ weights
      float *w = reinterpret_cast<float *>(smem + L::oW) + ((k & 1) * kRows + 16 * wm) * kTile;
      // of a warp: the least weight in rows without enough that count; bit 0: a
      // weight past the reference, bit 1: held in float32, bit 2: there is such a
      // least weight
      uint2 *tell = reinterpret_cast<uint2 *>(smem + L::oTell) + (k & 1) * L::kWarps;
      float sum[2], now[2] = {weighty[0], weighty[1]};
      {
        float over = 0.0f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          // a row that has seen nothing yet has no reference: whatever it sees now
          // is past the lowest float, and the turn begins again with a reference
          const float from = ref[b] == -INFINITY ? -3.402823466e38f : ref[b] - kUp;
          sum[b] = 0.0f;
#pragma unroll
          for (int j = 0; j < kOwn; ++j) {
            s[b][j] = exp2_approx(s[b][j] - from);
            sum[b] += s[b][j];
            over = fmaxf(over, s[b][j]);
          }
        }
        // weights that count, until a row has enough of them
        float least = kPast;
        if (__any_sync(0xffffffffu, fminf(weighty[0], weighty[1]) < kWeightyMin)) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float many = 0.0f, small = kPast;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
              many += s[b][j] < kWeighty ? 0.0f : 1.0f;  // NaN counts
              small = fminf(small, s[b][j] > 0.0f ? s[b][j] : kPast);
            }
            many += __shfl_xor_sync(0xffffffffu, many, 1);
            many += __shfl_xor_sync(0xffffffffu, many, 2);
            now[b] += many;
            if (now[b] < kWeightyMin) least = fminf(least, small);
          }
          least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(least)));
        }
        const bool few = least < kWeighty;
        const bool past = __any_sync(0xffffffffu, over > kPast);
        if (lane == 0) tell[warp] = make_uint2(__float_as_uint(least), (past ? 1u : 0u) | (few ? 2u : 0u) | (least < kPast ? 4u : 0u));
        // the 16-byte chunks of odd rows are stored with bit 2 of their index
        // flipped; a chunk is 4 weights, or their first parts, then the second
        const int col = (wb * L::kKeys + kOwn * t) ^ ((g & 1) << 4);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float *dst = w + (8 * b + g) * kTile + col;
          if constexpr (kNT == 2) {
            if (few) {
              *reinterpret_cast<float4 *>(dst) = make_float4(s[b][0], s[b][1], s[b][2], s[b][3]);
            } else {
              uint4 h;
              split_half2(s[b][0], s[b][1], h.x, h.z);
              split_half2(s[b][2], s[b][3], h.y, h.w);
              *reinterpret_cast<uint4 *>(dst) = h;
            }
          } else {
            if (few) {
              *reinterpret_cast<float2 *>(dst) = make_float2(s[b][0], s[b][1]);
            } else {
              uint32_t h0, h1;
              split_half2(s[b][0], s[b][1], h0, h1);
              uint32_t *u = reinterpret_cast<uint32_t *>(dst - 2 * (t & 1)) + (t & 1);
              u[0] = h0;
              u[2] = h1;
            }
          }
        }
      }
      __syncthreads();
      // every warp is past the values of the tile before: its stage is free
      const uint2 told = tell[lane % L::kWarps];
      fresh = false;
      uint32_t wide = 0;  // bit c: warp c of the row group holds its weights in float32
      float apart = kApart;
      if (__any_sync(0xffffffffu, told.y)) {
        fresh = __any_sync(0xffffffffu, told.y & 1);
        wide = __ballot_sync(0xffffffffu, told.y & 2) >> (wm * NB) & ((1u << NB) - 1);
        // nor may one bring a weight of a row without enough that count below what counts
        const uint32_t least = __reduce_min_sync(0xffffffffu, lane % L::kWarps / NB == wm ? told.x : 0x7f800000u);
        apart = fmaxf(apart, __fdividef(kWeighty, __uint_as_float(least)));
      }
      if (fresh) {
        __syncthreads();  // `tell` and the maxima are written again
        continue;
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        l_run[b] += sum[b];
        weighty[b] = now[b];
      }
      if (warp == 0) {
        load();
        look_ahead();
      }
      const float new_unit = exp2i(min(max(15 - static_cast<int>(largest >> 10), -15), 15));
      const float moved = new_unit * (1.0f / unit);
      unit = new_unit;
      const bool slow = wide || !(half_value(largest) * apart <= half_value(smallest));  // float32, too
      const bool special = tile * kTile + kTile > it.len;
      // ------------------------------------------------------------ values
      // The tile's products go to accumulators of their own: the tensor cores
      // round every sum towards zero, which over a long context would add up.
      float acc[4][4] = {};
      const uint8_t *vt = smem + L::oStage + st * L::kStageBytes + kTile * kRow;
      // A operands of 16 positions: the lane's 4 are 16 kg + 4 t ..., of rows g
      // and g + 8; B operands: column n of MMA tile j is element 4 n + j of the
      // block.
      if (!slow) {
        const __half2 unit2 = __float2half2_rn(unit);
#pragma unroll
        for (int kg = 0; kg < kTile / 16; ++kg) {
          const uint8_t *r = vt + (16 * kg + 4 * t) * kRow;
          uint32_t cw[4], f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            cw[j] = *reinterpret_cast<const uint32_t *>(r + j * kRow + kD / 16 + 32 * wb + 4 * g) ^ 0x80808080u;
            f[j] = *reinterpret_cast<const unsigned short *>(r + j * kRow + 2 * wb);
          }
          const int col = (16 * kg + 4 * t) ^ ((g & 1) << 4);
          const uint4 x0 = *reinterpret_cast<const uint4 *>(w + g * kTile + col);
          const uint4 x1 = *reinterpret_cast<const uint4 *>(w + (8 + g) * kTile + col);
          if (special) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = (f[j] & 0x7c00u) == 0x7c00u ? 0u : f[j];
          }
          const __half2 d01 = __hmul2(as_half2(__byte_perm(f[0], f[1], 0x5410)), unit2);
          const __half2 d23 = __hmul2(as_half2(__byte_perm(f[2], f[3], 0x5410)), unit2);
          auto times = [](uint32_t h, uint32_t l, __half2 d, uint32_t &hi, uint32_t &lo) {
            const __half2 y = __hmul2(as_half2(h), d);
            hi = as_bits(y);
            lo = as_bits(__hfma2(as_half2(l), d, __hfma2(as_half2(h), d, __hneg2(y))));
          };
          uint4 hi, lo;
          times(x0.x, x0.z, d01, hi.x, lo.x);
          times(x1.x, x1.z, d01, hi.y, lo.y);
          times(x0.y, x0.w, d23, hi.z, lo.z);
          times(x1.y, x1.w, d23, hi.w, lo.w);
          const uint32_t a = __byte_perm(cw[0], cw[1], 0x5140), b = __byte_perm(cw[0], cw[1], 0x7362);
          const uint32_t c = __byte_perm(cw[2], cw[3], 0x5140), e = __byte_perm(cw[2], cw[3], 0x7362);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v0 = codes_to_half2(j < 2 ? a : b, j & 1 ? 0x4342 : 0x4140);
            const uint32_t v1 = codes_to_half2(j < 2 ? c : e, j & 1 ? 0x4342 : 0x4140);
            mma_f16(acc[j], hi, v0, v1);
            mma_f16(acc[j], lo, v0, v1);
          }
        }
      } else {
#pragma unroll 2
        for (int kg = 0; kg < kTile / 16; ++kg) {
          const uint8_t *r = vt + (16 * kg + 4 * t) * kRow;
          const int col = (16 * kg + 4 * t) ^ ((g & 1) << 4);
          const uint4 x0 = *reinterpret_cast<const uint4 *>(w + g * kTile + col);
          const uint4 x1 = *reinterpret_cast<const uint4 *>(w + (8 + g) * kTile + col);
          float y0[4] = {__uint_as_float(x0.x), __uint_as_float(x0.y), __uint_as_float(x0.z), __uint_as_float(x0.w)};
          float y1[4] = {__uint_as_float(x1.x), __uint_as_float(x1.y), __uint_as_float(x1.z), __uint_as_float(x1.w)};
          if (!(wide >> (kNT == 2 ? kg : 2 * kg + (t >> 1)) & 1)) {  // held as two parts
            auto whole = [](uint32_t h, uint32_t l, float *y) {
              const float2 a = __half22float2(as_half2(h)), b = __half22float2(as_half2(l));
              y[0] = a.x + b.x;
              y[1] = a.y + b.y;
            };
            whole(x0.x, x0.z, y0);
            whole(x0.y, x0.w, y0 + 2);
            whole(x1.x, x1.z, y1);
            whole(x1.y, x1.w, y1 + 2);
          }
          uint32_t cw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            cw[j] = *reinterpret_cast<const uint32_t *>(r + j * kRow + kD / 16 + 32 * wb + 4 * g);
            const float d = f16_at(r + j * kRow + 2 * wb) * unit;
            // a weight of 0 (a masked position) stays 0 whatever the factor
            y0[j] = y0[j] != 0.0f ? y0[j] * d : 0.0f;
            y1[j] = y1[j] != 0.0f ? y1[j] * d : 0.0f;
          }
          uint4 p1, p2, p3;
          split_bf162(y0[0], y0[1], p1.x, p2.x, p3.x);
          split_bf162(y1[0], y1[1], p1.y, p2.y, p3.y);
          split_bf162(y0[2], y0[3], p1.z, p2.z, p3.z);
          split_bf162(y1[2], y1[3], p1.w, p2.w, p3.w);
          const uint32_t a = __byte_perm(cw[0], cw[1], 0x5140), b = __byte_perm(cw[0], cw[1], 0x7362);
          const uint32_t c = __byte_perm(cw[2], cw[3], 0x5140), e = __byte_perm(cw[2], cw[3], 0x7362);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v0 = codes_to_bf162(j < 2 ? a : b, j & 1 ? 0x4342 : 0x4140);
            const uint32_t v1 = codes_to_bf162(j < 2 ? c : e, j & 1 ? 0x4342 : 0x4140);
            mma_bf16(acc[j], p1, v0, v1);
            mma_bf16(acc[j], p2, v0, v1);
            mma_bf16(acc[j], p3, v0, v1);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][c] = fmaf(o[j][c], moved, acc[j][c]);
      ++tile;
      ++k;
    }

    // -------------------------------------------------------------- the item's rows
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float l = l_run[b];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (t == 0) sums[wb * kRows + 16 * wm + 8 * b + g] = l;
    }
    __syncthreads();
    const bool whole = first == 0 && last == it.tiles;
    float *part = p.parts + (2ll * blockIdx.x + (x0 == begin ? 0 : 1)) * L::kPart;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int r = 16 * wm + 8 * b + g;
      if (r >= n_rows) continue;
      float l = 0.0f;
#pragma unroll
      for (int c = 0; c < NB; ++c) l += sums[c * kRows + r];
      const int row = it.rt * kRows + r;
      float f = 1.0f / unit;  // a power of two
      float *dst = part + r * (kD + 4);
      if (whole) {
        f = l != 0.0f ? f / l : 0.0f;
        dst = out_row(p, it.s, it.h, row);
      } else if (wb == 0 && t == 0) {
        *reinterpret_cast<float2 *>(dst + kD) = make_float2(ref[b], l);
      }
      // the lane's 8 columns 8 t ... of the warp's block
      float4 *d4 = reinterpret_cast<float4 *>(dst + 32 * wb + 8 * t);
      d4[0] = make_float4(o[0][2 * b] * f, o[1][2 * b] * f, o[2][2 * b] * f, o[3][2 * b] * f);
      d4[1] = make_float4(o[0][2 * b + 1] * f, o[1][2 * b + 1] * f, o[2][2 * b + 1] * f, o[3][2 * b + 1] * f);
    }
  }
  // after a wait that gave up: the copies in flight land before the CTA ends
  if (!ok && tid == 0)
    for (uint32_t i = load_k > kStages ? load_k - kStages : 0; i < load_k; ++i)
      mbar_wait(&full[i % kStages], (i / kStages) & 1, p.err, DEVERR_DRAIN_WAIT, i);
}

constexpr size_t kHeadBytes = 8 * (kMaxSeq + 8);

// rows of a row tile for `rows` rows per key/value head (tokens times group)
inline int tile_rows(int rows) { return rows <= 16 ? 16 : 32; }

template <int NB, int WM>
cudaError_t launch_tree(const TreeParams &p, const DeviceInfo &dev, cudaStream_t s) {
  using L = Plan<NB, WM>;
  auto k = tree_kernel<NB, WM>;
  static LaunchOnce once;
  int per_sm = 0;
  cudaError_t e = once.prepare(dev.device, k, L::kThreads, L::kSmem, false, &per_sm);
  if (e != cudaSuccess) return e;
  const int grid = std::min(kMaxCtas, dev.sm_count * per_sm);
  e = launch_pdl(k, dim3(grid), dim3(L::kThreads), L::kSmem, s, p);
  if (e != cudaSuccess) return e;
  return launch_join<L::kD, L::kRows>(p, grid, s);
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" size_t epq_attention_tree_workspace_bytes(const epq_pages *pages, int n_heads, int ntok) {
  if (!pages_sizes_ok(pages) || n_heads < 1 || n_heads % pages->n_kv_heads ||
      n_heads / pages->n_kv_heads > kMaxGroupTree || ntok < 1 || ntok > kMaxTree)
    return 0;
  const int group = n_heads / pages->n_kv_heads;
  return kHeadBytes +
         2 * sizeof(float) * kMaxCtas * static_cast<size_t>(tile_rows(ntok * group)) * (pages->head_dim + 4);
}

extern "C" epq_status epq_attention_tree(const epq_pages *pages, int layer, const float *q, const float *k_new,
                                         const float *v_new, int n_heads, int ntok, float scale,
                                         const epq_attention_tree_opts *opts, float *out, void *ws, size_t ws_bytes,
                                         epq_stream_t stream) {
  TreeParams p = {};
  const epq_status st = pages_view(pages, &p.v);
  if (st != EPQ_OK) return st;
  if (!q || !k_new || !v_new || !out) return EPQ_ERR_ARG;
  const size_t need = epq_attention_tree_workspace_bytes(pages, n_heads, ntok);
  if (!need) return EPQ_ERR_SHAPE;
  if (layer < 0 || layer >= pages->n_layers) return EPQ_ERR_ARG;
  if (!(scale > 0.0f) || std::isinf(scale)) return EPQ_ERR_ARG;
  if (!ws || ws_bytes < need) return EPQ_ERR_WORKSPACE;
  const int D = pages->head_dim, n_kv = pages->n_kv_heads;
  p.q_ld = opts && opts->q_ld ? opts->q_ld : static_cast<int64_t>(n_heads) * D;
  p.kv_ld = opts && opts->kv_ld ? opts->kv_ld : static_cast<int64_t>(n_kv) * D;
  p.q_seq_ld = opts && opts->q_seq_ld ? opts->q_seq_ld : p.q_ld * ntok;
  p.kv_seq_ld = opts && opts->kv_seq_ld ? opts->kv_seq_ld : p.kv_ld * ntok;
  if (p.q_ld < 0 || p.kv_ld < 0 || p.q_seq_ld < 0 || p.kv_seq_ld < 0) return EPQ_ERR_SHAPE;
  if ((p.q_ld | p.kv_ld | p.q_seq_ld | p.kv_seq_ld) & 3) return EPQ_ERR_ALIGN;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(out) || !aligned16(ws))
    return EPQ_ERR_ALIGN;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  p.err = device_error_slot();
  if (!p.err) return EPQ_ERR_DEVICE;
  p.q = q;
  p.k_new = k_new;
  p.v_new = v_new;
  p.mask = opts ? opts->mask : nullptr;
  p.n_tok = opts ? opts->n_tok : nullptr;
  p.layer = layer;
  p.n_heads = n_heads;
  p.group = n_heads / n_kv;
  p.ntok = ntok;
  p.scale = scale;
  p.out = out;
  p.before = static_cast<long long *>(ws);
  p.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kHeadBytes);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool small = tile_rows(ntok * p.group) == 16;
  const cudaError_t e = D == 128 ? (small ? launch_tree<4, 1>(p, dev, s) : launch_tree<4, 2>(p, dev, s))
                                 : (small ? launch_tree<8, 1>(p, dev, s) : launch_tree<8, 2>(p, dev, s));
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
