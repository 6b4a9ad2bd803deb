// Attention of drafted tokens over a paged Q8_0 cache (epq_attention_tree).
//
//   s_ij = scale q_i . k_j,  o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// over the committed positions and the drafted tokens that token i's mask
// names.  The rows of one (sequence, key/value head) are its tokens times its
// `group` query heads (row r: token r / group, head r % group); a row tile is
// 16 MT of them.
//
// One pass over the positions in tiles of 64, a running maximum per row, and
// both products on the tensor cores (mma.sync m16n8k16, fp16 operands, float32
// sums) without giving up float32 accuracy:
//   scores   the int8 codes of a key are exact in fp16; a query row is scaled
//            by a power of two and split into two fp16 parts (2^-22 of the
//            entry, or 2^-38 of the row's largest); the sum of one 32-element
//            block is multiplied by that key's block factor in float32.
//   values   the codes are again the operand; the factor of (position, block)
//            goes to the other side: warp b owns the 32 columns of block b and
//            multiplies the weights by that block's factors before it splits
//            the product's 24 bits into three bf16 parts (exact, and with
//            float32's range: two fp16 parts would lose a weight below 2^-39
//            of the largest, which shows where the larger ones meet a code 0).
// Work: the tiles of all (sequence, head, row tile) items in a row, cut into
// equal shares, one per CTA.  A CTA's part of an item that it does not hold
// whole goes to the workspace (maximum, sum, unnormalised output), and a
// second launch joins the parts in the order of their positions.
// A producer warp streams the rows of a tile (contiguous within a page) with
// bulk copies into a ring of shared-memory stages; the D/32 consumer warps
// compute the scores of 64 / (D/32) positions each, exchange the weights
// through shared memory (one barrier per tile) and accumulate 32 columns each.
// The new rows are quantized into their tile by the CTAs that read it (the
// one of row tile 0 also stores them in the cache).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "pages.cuh"

namespace epq {
namespace {

constexpr int kMaxGroupTree = 16;
constexpr int kTile = 64;        // positions of a tile
constexpr int kStages = 3;
constexpr int kMaxCtas = 512;
constexpr int kJoinThreads = 128;

struct TreeParams {
  PagesView v;
  const float *q, *k_new, *v_new;
  const uint64_t *mask;
  const int32_t *n_tok;
  int64_t q_ld, q_seq_ld, kv_ld, kv_seq_ld;
  int layer, n_heads, group, ntok;
  float scale;
  float *out;
  float *parts;     // workspace: [2 per CTA][rows][D + 2]
  unsigned *err;
};

__device__ __forceinline__ int tree_size(const TreeParams &p, int s) {
  return p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok;
}

// Tiles of one row tile of a sequence with n tokens.
__device__ __forceinline__ int sequence_tiles(const TreeParams &p, int s, int n) {
  return n ? (seq_length(p.v, s) + n + kTile - 1) / kTile : 0;
}

__device__ __forceinline__ uint64_t token_mask(const TreeParams &p, int s, int i, int n) {
  const uint64_t m = p.mask ? p.mask[s * p.ntok + i] : ~0ull >> (63 - i);
  return n >= 64 ? m : m & ((1ull << n) - 1);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Codes: a byte u = code + 128 under the exponent byte 0x64 is the half 1024 + u.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t x, uint32_t sel) {
  const uint32_t h = __byte_perm(x, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t *>(&r);
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

__device__ __forceinline__ float f16_at(const uint8_t *p) {
  return __half2float(__ushort_as_half(*reinterpret_cast<const unsigned short *>(p)));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// x, y -> fp16 parts: first = rounded, second = the rest rounded.
__device__ __forceinline__ void split_half2(float x, float y, uint32_t &first, uint32_t &rest) {
  first = pack_half2(x, y);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&first));
  rest = pack_half2(x - f.x, y - f.y);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What a work item is: rows [16 MT rt, ...) of head h of sequence s.
struct Item {
  int s, h, rt, tiles, len, n;
};

template <int NB, int MT>
struct Plan {
  static constexpr int kD = 32 * NB;
  static constexpr int kRow = kD + kD / 16;
  static constexpr int kRows = 16 * MT;
  static constexpr int kConsumers = 32 * NB;
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kKeys = kTile / NB;  // positions whose scores a warp computes
  static constexpr int kNT = kKeys / 8;
  static constexpr uint32_t kStageBytes = 2u * kTile * kRow;
  // shared memory (bytes)
  static constexpr uint32_t oStage = 0;
  static constexpr uint32_t oQ = oStage + kStages * kStageBytes;       // query fragments, two parts
  static constexpr uint32_t oW = oQ + 2u * 2u * kRows * kD;            // [2][rows][64] weights
  static constexpr uint32_t oMax = oW + 2u * 4u * kRows * kTile;       // [2][NB][rows] tile maxima
  static constexpr uint32_t oSum = oMax + 2u * 4u * NB * kRows;        // [NB][rows]
  static constexpr uint32_t oMask = oSum + 4u * NB * kRows;            // [rows] mask words
  static constexpr uint32_t oScale = oMask + 8u * kRows;               // [rows] score factors (log2 units)
  static constexpr uint32_t oTiles = oScale + 4u * kRows;              // [n_seq + 1] tiles before a sequence
  static constexpr uint32_t oBar = oTiles + 8u * (kMaxSeq + 8);        // full, empty
  static constexpr uint32_t oMiss = oBar + 16u * kStages;              // [stages] missing pieces
  static constexpr uint32_t kSmem = oMiss + 4u * kStages + 4u;
};

template <int NB, int MT>
__global__ void __launch_bounds__(Plan<NB, MT>::kThreads, NB == 4 ? (MT == 1 ? 3 : 2) : 1) tree_kernel(const __grid_constant__ TreeParams p) {
  using L = Plan<NB, MT>;
  constexpr int kRows = L::kRows, kD = L::kD, kRow = L::kRow, kNT = L::kNT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::oBar);
  uint64_t *empty = full + kStages;
  long long *before = reinterpret_cast<long long *>(smem + L::oTiles);
  unsigned *miss = reinterpret_cast<unsigned *>(smem + L::oMiss);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NB);
    }
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  // tiles before each sequence
  auto rows_tiles = [&](int s, int *nrt) {
    const int n = tree_size(p, s);
    *nrt = (n * p.group + kRows - 1) / kRows;
    return sequence_tiles(p, s, n);
  };
  for (int s = tid; s < p.v.n_seq; s += L::kThreads) {
    int nrt;
    const int tiles = rows_tiles(s, &nrt);
    before[s + 1] = static_cast<long long>(tiles) * nrt * p.v.n_kv;
  }
  if (tid == 0) before[0] = 0;
  __syncthreads();
  if (warp == 0) {
    long long run = 0;
    for (int s0 = 0; s0 < p.v.n_seq; s0 += 32) {
      long long x = s0 + lane < p.v.n_seq ? before[s0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (s0 + lane < p.v.n_seq) before[s0 + lane + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const long long total = before[p.v.n_seq];
  const long long ctas = gridDim.x < total ? gridDim.x : total;
  // tokens beyond a sequence's tree: 0
  for (int r = blockIdx.x; r < p.v.n_seq * p.ntok; r += gridDim.x) {
    if (r % p.ntok < tree_size(p, r / p.ntok)) continue;
    float4 *o = reinterpret_cast<float4 *>(p.out + static_cast<int64_t>(r) * p.n_heads * kD);
    for (int i = tid; i < p.n_heads * kD / 4; i += L::kThreads) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (blockIdx.x >= ctas) return;
  const long long begin = blockIdx.x * total / ctas, end = (blockIdx.x + 1) * total / ctas;
  // the item that holds tile x, and the tile's place in it
  auto find = [&](long long x, Item &it) {
    int lo = 0, hi = p.v.n_seq - 1;
    while (lo < hi) {  // the last sequence with before[s] <= x (empty ones are passed over)
      const int mid = (lo + hi + 1) / 2;
      if (before[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    int nrt;
    it.s = lo;
    it.tiles = rows_tiles(lo, &nrt);
    it.len = seq_length(p.v, lo);
    it.n = tree_size(p, lo);
    const long long rel = x - before[lo];
    const int k = static_cast<int>(rel / it.tiles);
    it.h = k / nrt;
    it.rt = k % nrt;
    return static_cast<int>(rel % it.tiles);
  };
  const int piece_rows = min(p.v.P, kTile);

  // ================================================================ producer
  if (warp == NB) {
    bool ok = true;
    uint32_t k = 0;
    for (long long x = begin; x < end;) {
      Item it;
      const int first = find(x, it);
      const int last = static_cast<int>(min(static_cast<long long>(it.tiles), first + (end - x)));
      x += last - first;
      for (int tile = first; tile < last; ++tile, ++k) {
        const int st = k % kStages;
        if (k >= kStages && ok)
          ok = warp_wait(&empty[st], (k / kStages - 1) & 1, p.err, DEVERR_EMPTY_WAIT, k);
        // lane = 2 * piece + plane
        const int piece = lane >> 1, c = lane & 1;
        const int pos = tile * kTile + piece * piece_rows;
        const int rows = piece < kTile / piece_rows ? min(max(it.len - pos, 0), piece_rows) : 0;
        const int page = rows > 0 ? seq_page(p.v, it.s, pos / p.v.P) : 0;
        const uint32_t bytes = rows > 0 && page >= 0 ? (static_cast<uint32_t>(rows) * kRow) & ~15u : 0u;
        const unsigned lost = __ballot_sync(0xffffffffu, page < 0);
        if (lost && lane == 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(it.s));
        const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0) {
          miss[st] = lost;
          if (all) mbar_arrive_expect_tx(&full[st], all);
          else mbar_arrive(&full[st]);
        }
        __syncwarp();
        if (bytes)
          bulk_g2s(smem + L::oStage + st * L::kStageBytes + (c * kTile + piece * piece_rows) * kRow,
                   page_row(p.v, p.layer, page, it.h, c, pos % p.v.P), bytes, &full[st]);
      }
    }
    // every copy has landed before the CTA ends
    for (uint32_t i = k > kStages ? k - kStages : 0; i < k; ++i)
      warp_wait(&full[i % kStages], (i / kStages) & 1, p.err, DEVERR_DRAIN_WAIT, i);
    return;
  }

  // ================================================================ consumers
  auto sync = [&]() { named_sync(1, L::kConsumers); };
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
    x += last - first;
    const int n_rows = min(kRows, it.n * p.group - it.rt * kRows);

    // -------------------------------------------------------------- queries
    // A warp takes a row: scaled by a power of two so that the largest entry
    // is in [2^13, 2^14), split, stored as MMA A fragments (element 16 ks +
    // 4 t + e of a block pair: lane t of the row, register e / 2).
    for (int r = warp; r < kRows; r += NB) {
      const int row = it.rt * kRows + r, i = row / p.group;
      float4 q[NB / 4];
      float a = 0.0f;
#pragma unroll
      for (int c = 0; c < NB / 4; ++c) {
        q[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n_rows)
          q[c] = *reinterpret_cast<const float4 *>(p.q + it.s * p.q_seq_ld + i * p.q_ld +
                                                   (it.h * p.group + row % p.group) * kD + 128 * c + 4 * lane);
        a = fmaxf(fmaxf(a, fmaxf(fabsf(q[c].x), fabsf(q[c].y))), fmaxf(fabsf(q[c].z), fabsf(q[c].w)));
      }
      a = warp_absmax(a);
      const int e = min(max(static_cast<int>(__float_as_uint(a) >> 23) - 127, -100), 127);
      const float up = exp2i(13 - e);
      if (lane == 0) {
        row_scale[r] = p.scale * 1.4426950408889634f * exp2i(e - 13);
        row_mask[r] = r < n_rows ? token_mask(p, it.s, i, it.n) : 0;
      }
#pragma unroll
      for (int c = 0; c < NB / 4; ++c) {
        uint32_t h0, h1, l0, l1;
        split_half2(q[c].x * up, q[c].y * up, h0, l0);
        split_half2(q[c].z * up, q[c].w * up, h1, l1);
        // float4 index 32 c + lane = 4 (16-element step) + t
        const int step = 8 * c + (lane >> 2);
        uint32_t *f = reinterpret_cast<uint32_t *>(smem + L::oQ) +
                      (((r >> 4) * (2 * NB) + step) * 2 * 32 + (r & 7) * 4 + t) * 4 + ((r >> 3) & 1);
        f[0] = h0;
        f[2] = h1;
        f[128] = l0;
        f[130] = l1;
      }
    }
    sync();

    float o[MT][4][4] = {};
    float m_run[MT][2], l_run[MT][2], c_row[MT][2];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        m_run[a][b] = -INFINITY;
        l_run[a][b] = 0.0f;
        c_row[a][b] = row_scale[16 * a + 8 * b + g];
      }
    float s[MT][2][2 * kNT];  // scores of rows g, g + 8 at the lane's 2 kNT positions

    // Scores of tile `tile` (pipeline step kk) into s, its row maxima into oMax.
    auto scores = [&](int tile, uint32_t kk) {
      const int st = kk % kStages;
      uint8_t *kt = smem + L::oStage + st * L::kStageBytes, *vt = kt + kTile * kRow;
      if (ok) ok = warp_wait(&full[st], (kk / kStages) & 1, p.err, DEVERR_FULL_WAIT, kk);
      const int t0 = tile * kTile;
      const unsigned lost = miss[st];
      const bool special = t0 + kTile > it.len || lost;
      if (special) {
        // new rows, the end of an odd number of committed rows (a bulk copy
        // moves 16 bytes), and rows that hold nothing (their factors are 0)
        for (int rr = warp; rr < 2 * kTile; rr += NB) {
          const int r = rr >> 1, c = rr & 1, pos = t0 + r;
          uint8_t *dst = (c ? vt : kt) + r * kRow;
          const bool gone = lost >> (2 * (r / piece_rows)) & 1;
          if (pos < it.len && !gone) {
            if (pos == it.len - 1 && ((r % piece_rows + 1) * kRow & 8) && lane == 0)
              *reinterpret_cast<uint2 *>(dst + kRow - 8) = *reinterpret_cast<const uint2 *>(
                  page_row(p.v, p.layer, seq_page(p.v, it.s, pos / p.v.P), it.h, c, pos % p.v.P) + kRow - 8);
          } else if (pos >= it.len && pos < it.len + it.n) {
            const int i = pos - it.len;
            uint8_t *row = nullptr;
            if (it.rt == 0) {
              const int page = seq_page(p.v, it.s, pos / p.v.P);
              if (page >= 0) row = page_row(p.v, p.layer, page, it.h, c, pos % p.v.P);
              else if (lane == 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(it.s));
            }
            const float *src = (c ? p.v_new : p.k_new) + it.s * p.kv_seq_ld + i * p.kv_ld + it.h * kD;
#pragma unroll
            for (int q4 = 0; q4 < NB / 4; ++q4) {
              // Q8_0 with the packer's arithmetic (factor fp16(max|x| / 127),
              // codes rint(x / factor) in +-127, 0 for a zero factor); 8 lanes
              // hold a block
              const float4 xv = *reinterpret_cast<const float4 *>(src + 128 * q4 + 4 * lane);
              const float e[4] = {__fadd_rn(xv.x, 0.0f), __fadd_rn(xv.y, 0.0f), __fadd_rn(xv.z, 0.0f),
                                  __fadd_rn(xv.w, 0.0f)};
              float a = fmaxf(fmaxf(fabsf(e[0]), fabsf(e[1])), fmaxf(fabsf(e[2]), fabsf(e[3])));
#pragma unroll
              for (int w = 1; w < 8; w <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, w));
              const __half dh = __float2half_rn(__fdiv_rn(a, 127.0f));
              const float d = __half2float(dh);
              uint32_t word = 0;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float y = d != 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(e[j], d)), -127.0f), 127.0f) : 0.0f;
                word |= (static_cast<uint32_t>(static_cast<int>(y)) & 0xffu) << (8 * j);
              }
              const int at = kD / 16 + 128 * q4 + 4 * lane, fat = 2 * (4 * q4 + (lane >> 3));
              *reinterpret_cast<uint32_t *>(dst + at) = word;
              if ((lane & 7) == 0) *reinterpret_cast<uint16_t *>(dst + fat) = __half_as_ushort(dh);
              if (row) {
                *reinterpret_cast<uint32_t *>(row + at) = word;
                if ((lane & 7) == 0) *reinterpret_cast<uint16_t *>(row + fat) = __half_as_ushort(dh);
              }
            }
          } else if (lane < NB) {
            reinterpret_cast<uint16_t *>(dst)[lane] = 0;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        sync();
      }
      const uint8_t *kw = kt + warp * L::kKeys * kRow;
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int j = 0; j < 2 * kNT; ++j) s[a][0][j] = s[a][1][j] = 0.0f;
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
        float d[2 * kNT];  // factors of the lane's positions 2 kNT t ...
#pragma unroll
        for (int j = 0; j < 2 * kNT; ++j) d[j] = f16_at(kw + (2 * kNT * t + j) * kRow + 2 * b);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          float acc[kNT][4] = {};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const uint4 *f = reinterpret_cast<const uint4 *>(smem + L::oQ) + (a * (2 * NB) + 2 * b + ks) * 64 + lane;
            const uint4 hi = f[0], lo = f[32];
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
              mma_f16(acc[j], hi, kb[j][2 * ks], kb[j][2 * ks + 1]);
              mma_f16(acc[j], lo, kb[j][2 * ks], kb[j][2 * ks + 1]);
            }
          }
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            s[a][0][j] = fmaf(d[j], acc[j][0], s[a][0][j]);
            s[a][0][kNT + j] = fmaf(d[kNT + j], acc[j][1], s[a][0][kNT + j]);
            s[a][1][j] = fmaf(d[j], acc[j][2], s[a][1][j]);
            s[a][1][kNT + j] = fmaf(d[kNT + j], acc[j][3], s[a][1][kNT + j]);
          }
        }
      }
      float *mx = reinterpret_cast<float *>(smem + L::oMax) + ((kk & 1) * NB + warp) * kRows;
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float m = -INFINITY;
          const uint64_t may = special ? row_mask[16 * a + 8 * b + g] : 0;
#pragma unroll
          for (int j = 0; j < 2 * kNT; ++j) {
            s[a][b][j] *= c_row[a][b];
            if (special) {
              const int r = warp * L::kKeys + 2 * kNT * t + j, i = t0 + r - it.len;
              const bool see = i < 0 ? !(lost >> (2 * (r / piece_rows)) & 1) : i < 64 && (may >> i & 1);
              if (!see) s[a][b][j] = -INFINITY;
            }
            m = fmaxf(m, s[a][b][j]);
          }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if (t == 0) mx[16 * a + 8 * b + g] = m;
        }
    };

    scores(first, k);
    sync();
    for (int tile = first; tile < last; ++tile, ++k) {
      const int st = k % kStages;
      // ------------------------------------------------------------ weights
      float keep[MT][2];
      float *w = reinterpret_cast<float *>(smem + L::oW) + (k & 1) * kRows * kTile;
      {
        const float *mx = reinterpret_cast<const float *>(smem + L::oMax) + (k & 1) * NB * kRows;
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int r = 16 * a + 8 * b + g;
            float m = m_run[a][b];
#pragma unroll
            for (int c = 0; c < NB; ++c) m = fmaxf(m, mx[c * kRows + r]);
            const float ref = m == -INFINITY ? 0.0f : m;
            keep[a][b] = exp2_approx(m_run[a][b] - ref);
            m_run[a][b] = m;
            float sum = 0.0f, e[2 * kNT];
#pragma unroll
            for (int j = 0; j < 2 * kNT; ++j) {
              e[j] = exp2_approx(s[a][b][j] - ref);
              sum += e[j];
            }
            l_run[a][b] = fmaf(l_run[a][b], keep[a][b], sum);
            // the 16-byte chunks of odd rows are stored with bit 2 of their index flipped
            const int col = warp * L::kKeys + 2 * kNT * t;
            float *dst = w + r * kTile + (col ^ ((g & 1) << 4));
            if constexpr (kNT == 2) *reinterpret_cast<float4 *>(dst) = make_float4(e[0], e[1], e[2], e[3]);
            else *reinterpret_cast<float2 *>(dst) = make_float2(e[0], e[1]);
          }
      }
      if (tile + 1 < last) scores(tile + 1, k + 1);
      sync();
      // ------------------------------------------------------------ values
      // The tile's products go to accumulators of their own: the tensor cores
      // round every sum towards zero, which over a long context would add up.
      float acc[MT][4][4] = {};
      const uint8_t *vt = smem + L::oStage + st * L::kStageBytes + kTile * kRow;
      const bool special = tile * kTile + kTile > it.len;  // a new row's factor may not be finite
#pragma unroll
      for (int kg = 0; kg < kTile / 16; ++kg) {
        const uint8_t *r = vt + (16 * kg + 4 * t) * kRow;
        const uint32_t w0 = *reinterpret_cast<const uint32_t *>(r + kD / 16 + 32 * warp + 4 * g);
        const uint32_t w1 = *reinterpret_cast<const uint32_t *>(r + kRow + kD / 16 + 32 * warp + 4 * g);
        const uint32_t w2 = *reinterpret_cast<const uint32_t *>(r + 2 * kRow + kD / 16 + 32 * warp + 4 * g);
        const uint32_t w3 = *reinterpret_cast<const uint32_t *>(r + 3 * kRow + kD / 16 + 32 * warp + 4 * g);
        float d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = f16_at(r + j * kRow + 2 * warp);
        // column n of MMA tile j: element 4 n + j of the block
        uint32_t vb[4][2];
        {
          const uint32_t a = __byte_perm(w0, w1, 0x5140), b = __byte_perm(w0, w1, 0x7362);
          const uint32_t c = __byte_perm(w2, w3, 0x5140), e = __byte_perm(w2, w3, 0x7362);
          vb[0][0] = codes_to_bf162(a, 0x4140);
          vb[1][0] = codes_to_bf162(a, 0x4342);
          vb[2][0] = codes_to_bf162(b, 0x4140);
          vb[3][0] = codes_to_bf162(b, 0x4342);
          vb[0][1] = codes_to_bf162(c, 0x4140);
          vb[1][1] = codes_to_bf162(c, 0x4342);
          vb[2][1] = codes_to_bf162(e, 0x4140);
          vb[3][1] = codes_to_bf162(e, 0x4342);
        }
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          uint4 p1, p2, p3;
          const int col = (16 * kg + 4 * t) ^ ((g & 1) << 4);
          float4 x0 = *reinterpret_cast<const float4 *>(w + (16 * a + g) * kTile + col);
          float4 x1 = *reinterpret_cast<const float4 *>(w + (16 * a + 8 + g) * kTile + col);
          if (special) {
            x0 = make_float4(x0.x != 0.0f ? x0.x * d[0] : 0.0f, x0.y != 0.0f ? x0.y * d[1] : 0.0f,
                             x0.z != 0.0f ? x0.z * d[2] : 0.0f, x0.w != 0.0f ? x0.w * d[3] : 0.0f);
            x1 = make_float4(x1.x != 0.0f ? x1.x * d[0] : 0.0f, x1.y != 0.0f ? x1.y * d[1] : 0.0f,
                             x1.z != 0.0f ? x1.z * d[2] : 0.0f, x1.w != 0.0f ? x1.w * d[3] : 0.0f);
          } else {
            x0 = make_float4(x0.x * d[0], x0.y * d[1], x0.z * d[2], x0.w * d[3]);
            x1 = make_float4(x1.x * d[0], x1.y * d[1], x1.z * d[2], x1.w * d[3]);
          }
          split_bf162(x0.x, x0.y, p1.x, p2.x, p3.x);
          split_bf162(x1.x, x1.y, p1.y, p2.y, p3.y);
          split_bf162(x0.z, x0.w, p1.z, p2.z, p3.z);
          split_bf162(x1.z, x1.w, p1.w, p2.w, p3.w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_bf16(acc[a][j], p1, vb[j][0], vb[j][1]);
            mma_bf16(acc[a][j], p2, vb[j][0], vb[j][1]);
            mma_bf16(acc[a][j], p3, vb[j][0], vb[j][1]);
          }
        }
      }
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[a][j][c] = fmaf(o[a][j][c], keep[a][c >> 1], acc[a][j][c]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // -------------------------------------------------------------- the item's rows
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float l = l_run[a][b];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) sums[warp * kRows + 16 * a + 8 * b + g] = l;
      }
    sync();
    const bool whole = first == 0 && last == it.tiles;
    float *part = p.parts + (2ll * blockIdx.x + (x0 == begin ? 0 : 1)) * kRows * (kD + 2);
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = 16 * a + 8 * b + g;
        if (r >= n_rows) continue;
        float l = 0.0f;
#pragma unroll
        for (int c = 0; c < NB; ++c) l += sums[c * kRows + r];
        const int row = it.rt * kRows + r;
        float f = 1.0f;
        float *dst = part + r * (kD + 2);
        if (whole) {
          f = l != 0.0f ? 1.0f / l : 0.0f;
          dst = p.out + (static_cast<int64_t>(it.s) * p.ntok + row / p.group) * p.n_heads * kD +
                (it.h * p.group + row % p.group) * kD;
        } else if (warp == 0 && t == 0) {
          dst[kD] = m_run[a][b];
          dst[kD + 1] = l;
        }
        // the lane's 8 columns 8 t ... of the warp's block
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y0 = o[a][j][2 * b], y1 = o[a][j][2 * b + 1];
          dst[32 * warp + 8 * t + j] = whole ? (l != 0.0f ? y0 * f : 0.0f) : y0;
          dst[32 * warp + 8 * t + 4 + j] = whole ? (l != 0.0f ? y1 * f : 0.0f) : y1;
        }
      }
  }
}

// Joins the parts of the items that more than one CTA holds: one warp per
// (item, row), the parts in the order of their positions.
template <int NB, int MT>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ TreeParams p, int grid) {
  constexpr int kRows = 16 * MT, kD = 32 * NB, kPart = kRows * (kD + 2);
  __shared__ long long before_s;
  __shared__ long long total_s;
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = tree_size(p, s);
  const int nrt = (n * p.group + kRows - 1) / kRows;
  const int tiles = sequence_tiles(p, s, n);
  // tiles of the sequences before this one, and of all
  if (warp == 0) {
    long long below = 0, all = 0;
    for (int k = lane; k < p.v.n_seq; k += 32) {
      const int m = tree_size(p, k);
      const long long x = static_cast<long long>(sequence_tiles(p, k, m)) * ((m * p.group + kRows - 1) / kRows) * p.v.n_kv;
      all += x;
      if (k < s) below += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      below += __shfl_xor_sync(0xffffffffu, below, o);
      all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (lane == 0) before_s = below, total_s = all;
  }
  __syncthreads();
  const int x = blockIdx.x * (kJoinThreads / 32) + warp;  // (head, row of the head)
  const int h = x / (p.ntok * p.group), row = x % (p.ntok * p.group);
  if (h >= p.v.n_kv || row >= n * p.group) return;
  const long long total = total_s, ctas = grid < total ? grid : total;
  const long long i0 = before_s + static_cast<long long>(h * nrt + row / kRows) * tiles, i1 = i0 + tiles - 1;
  const int c0 = static_cast<int>(((i0 + 1) * ctas - 1) / total), c1 = static_cast<int>(((i1 + 1) * ctas - 1) / total);
  if (c0 == c1) return;  // one CTA held it whole and wrote it
  // only the first of the item's CTAs can have begun before it
  const float *rest = p.parts + (row % kRows) * (kD + 2);
  const float *head = rest + (c0 * total / ctas >= i0 ? 0 : kPart);
  float top = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, (c == c0 ? head : rest)[2ll * c * kPart + kD]);
  top = warp_max_all(top);
  const float ref = top == -INFINITY ? 0.0f : top;
  float4 y[NB / 4] = {};
  float den = 0.0f;
#pragma unroll 8
  for (int c = c0; c <= c1; ++c) {
    const float *q = (c == c0 ? head : rest) + 2ll * c * kPart;
    const float2 ml = *reinterpret_cast<const float2 *>(q + kD);
    const float f = exp2f(ml.x - ref);  // 0 for a part that saw nothing
    den = fmaf(f, ml.y, den);
#pragma unroll
    for (int e = 0; e < NB / 4; ++e) {
      const float2 a = *reinterpret_cast<const float2 *>(q + 128 * e + 4 * lane);
      const float2 b = *reinterpret_cast<const float2 *>(q + 128 * e + 4 * lane + 2);
      y[e].x = fmaf(f, a.x, y[e].x);
      y[e].y = fmaf(f, a.y, y[e].y);
      y[e].z = fmaf(f, b.x, y[e].z);
      y[e].w = fmaf(f, b.y, y[e].w);
    }
  }
  float *out = p.out + (static_cast<int64_t>(s) * p.ntok + row / p.group) * p.n_heads * kD +
               (h * p.group + row % p.group) * kD;
#pragma unroll
  for (int e = 0; e < NB / 4; ++e)
    *reinterpret_cast<float4 *>(out + 128 * e + 4 * lane) =
        den != 0.0f ? make_float4(y[e].x / den, y[e].y / den, y[e].z / den, y[e].w / den) : make_float4(0.f, 0.f, 0.f, 0.f);
}

// rows of a row tile for ntok tokens of `group` heads
inline int tile_rows(int rows) { return rows <= 16 ? 16 : 32; }

template <int NB, int MT>
cudaError_t launch_tree(const TreeParams &p, const DeviceInfo &dev, cudaStream_t s) {
  using L = Plan<NB, MT>;
  auto k = tree_kernel<NB, MT>;
  static LaunchOnce once;
  int per_sm = 0;
  cudaError_t e = once.prepare(dev.device, k, L::kThreads, L::kSmem, false, &per_sm);
  if (e != cudaSuccess) return e;
  const int grid = std::min(kMaxCtas, dev.sm_count * per_sm);
  e = launch_pdl(k, dim3(grid), dim3(L::kThreads), L::kSmem, s, p);
  if (e != cudaSuccess) return e;
  const int rows = p.v.n_kv * p.ntok * p.group;
  return launch_pdl(join_kernel<NB, MT>, dim3((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32), p.v.n_seq),
                    dim3(kJoinThreads), 0, s, p, grid);
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" size_t epq_attention_tree_workspace_bytes(const epq_pages *pages, int n_heads, int ntok) {
  if (!pages_sizes_ok(pages) || n_heads < 1 || n_heads % pages->n_kv_heads ||
      n_heads / pages->n_kv_heads > kMaxGroupTree || ntok < 1 || ntok > kMaxTree)
    return 0;
  const int group = n_heads / pages->n_kv_heads;
  return 2 * sizeof(float) * kMaxCtas * static_cast<size_t>(tile_rows(ntok * group)) * (pages->head_dim + 2);
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
  p.parts = static_cast<float *>(ws);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool small = tile_rows(ntok * p.group) == 16;
  cudaError_t e = D == 128 ? (small ? launch_tree<4, 1>(p, dev, s) : launch_tree<4, 2>(p, dev, s))
                           : (small ? launch_tree<8, 1>(p, dev, s) : launch_tree<8, 2>(p, dev, s));
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
