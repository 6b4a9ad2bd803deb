// Rotary positions as the kernels see them: a token's position, the row of the
// table that holds its cosines and sines, and one turned element.
//
//   y0 = x0 c - x1 s,  y1 = x1 c + x0 s
//
// Products and sums are rounded one by one (no fused multiply-add), so that a
// key is quantized to the same codes wherever its rotation is computed.
#pragma once

#include "common.cuh"

namespace epq {

// Where token i of sequence s stands: given, or `start` and what comes before
// the token in its sequence (its index, or its ancestors in a tree).
struct Places {
  const int32_t *position, *start;
  const uint64_t *mask;
  const int32_t *n_tok;
  int ntok;
};

struct RotationView {
  const float *table;  // [n_pos][rot / 2][2]; null: nothing is rotated
  int64_t n_pos;
  int rot, first, interleaved;
};

// A null rotation is one that turns nothing.
inline epq_status rotation_view(const epq_rotation *r, int head_dim, RotationView *v) {
  *v = {};
  if (!r) return EPQ_OK;
  if (!r->table || r->n_pos < 1) return EPQ_ERR_ARG;
  if (r->n_pos > (int64_t(1) << 30) || r->rot_dim < 2 || r->rot_dim % 2 || r->first < 0 || r->first > head_dim ||
      r->rot_dim > head_dim - r->first)
    return EPQ_ERR_SHAPE;
  if (!aligned16(r->table)) return EPQ_ERR_ALIGN;
  *v = {r->table, r->n_pos, r->rot_dim, r->first, r->interleaved != 0};
  return EPQ_OK;
}

// Whether four elements at a multiple of 4 are turned by 16-byte reads alone:
// both elements of a pair, and the pair's cosine and sine, lie in them.
inline bool rotates_by_four(const RotationView &r) {
  return r.first % 4 == 0 && r.rot % (r.interleaved ? 4 : 8) == 0;
}

#ifdef __CUDACC__
__device__ __forceinline__ int tokens_of(const Places &p, int s) {
  return p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok;
}

__device__ __forceinline__ int64_t place_of(const Places &p, int s, int i) {
  const int64_t at = static_cast<int64_t>(s) * p.ntok + i;
  if (p.position) return p.position[at];
  const int64_t base = p.start ? p.start[s] : 0;
  if (!p.mask) return base + i;
  return base + __popcll(p.mask[at] & (~0ull >> (64 - p.ntok)) & ~(1ull << i));
}

// The table's row of a position, or null when it has none.
__device__ __forceinline__ const float *angles_at(const RotationView &r, int64_t place) {
  return place >= 0 && place < r.n_pos ? r.table + place * r.rot : nullptr;
}

// An element of a pair: `x` turned with its partner.  `up`: it is the second.
__device__ __forceinline__ float turned(float x, float partner, float c, float s, bool up) {
  const float a = __fmul_rn(x, c), b = __fmul_rn(partner, s);
  return up ? __fadd_rn(a, b) : __fsub_rn(a, b);
}
#endif

}  // namespace epq
