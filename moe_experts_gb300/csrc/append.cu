// Any number of new rows brought into a paged Q8_0 cache, the keys rotated on
// the way (epq_pages_append), and their commit (epq_pages_advance).
//
//   row = (d_b, c_e):  d_b = fp16(max_e |x_e| / 127),  c_e = rint(x_e / d_b)
//
// over blocks b of 32 elements, x the value, or the key after its rotation.
//
// 8192 tokens of 8 heads of 128 take 20.6 us, 4.3 TB/s of the 71 MB read and 18 MB
// written (0.64 of the copy rate): bound by the instructions of the quantization
// (0.74 issued per cycle of a scheduler when a row of 128 elements took some 125 of
// them; with the bound on a block's codes asked of each code it was 21.1 us).
// With an IEEE division for each element it was 36 us, with every head's position,
// page and angles worked out anew 33 us.  8 rows in a tree: 3.0 us, one chain of
// length, page, angles, store.
#include <algorithm>

#include "pages.cuh"
#include "rope.cuh"

namespace epq {
namespace {

constexpr int kWarps = 8;

struct AppendParams {
  PagesView v;
  RotationView r;
  Places p;
  const float *k, *x;  // keys and values
  int64_t ld, seq_ld;
  int layer;
  unsigned warps, groups, each;  // groups of `each` heads that a token has, and of all tokens
  unsigned page_bits, plane_bytes;
  unsigned *err;
};

// What turns elements e .. e + 3 of a head: y = x c + partner s, each product
// and the sum rounded (the sign of the formula's difference is in s).  kFour:
// pairs, cosines and sines lie in 16-byte words, and are the same for all heads.
struct Turn {
  float c[4], s[4];
  int partner;  // of the first element, relative to it; 1: the partners are among the four; 0: nothing is turned
};

__device__ __forceinline__ Turn turn_of(const RotationView &r, int e, const float *angles) {
  Turn t;
  const int at = e - r.first, half = r.rot / 2;
  t.partner = 0;
  if (!angles || at < 0 || at >= r.rot) return t;
  if (r.interleaved) {
    const float4 a = *reinterpret_cast<const float4 *>(angles + at);
    t.c[0] = t.c[1] = a.x, t.s[0] = -a.y, t.s[1] = a.y, t.c[2] = t.c[3] = a.z, t.s[2] = -a.w, t.s[3] = a.w;
    t.partner = 1;
  } else {
    const bool up = at >= half;
    const float *cs = angles + 2 * (up ? at - half : at);
    const float4 a = *reinterpret_cast<const float4 *>(cs), b = *reinterpret_cast<const float4 *>(cs + 4);
    t.c[0] = a.x, t.c[1] = a.z, t.c[2] = b.x, t.c[3] = b.z;
    t.s[0] = up ? a.y : -a.y, t.s[1] = up ? a.w : -a.w, t.s[2] = up ? b.y : -b.y, t.s[3] = up ? b.w : -b.w;
    t.partner = up ? -half : half;
  }
  return t;
}

// x: where the four elements `a` lie.
__device__ __forceinline__ float4 turned4(const Turn &t, const float *x, float4 a) {
  if (t.partner == 0) return a;
  float4 b = make_float4(a.y, a.x, a.w, a.z);
  if (t.partner != 1) b = *reinterpret_cast<const float4 *>(x + t.partner);
  const auto f = [&](float u, float v, int i) { return __fadd_rn(__fmul_rn(u, t.c[i]), __fmul_rn(v, t.s[i])); };
  return make_float4(f(a.x, b.x, 0), f(a.y, b.y, 1), f(a.z, b.z, 2), f(a.w, b.w, 3));
}

// The same where pairs lie anywhere: x is the head's row, `a` its elements e .. e + 3.
__device__ __forceinline__ float4 turned_any(const RotationView &r, const float *x, int e, const float *angles, float4 a) {
  const int half = r.rot / 2;
  float y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int i = e - r.first + n;
    if (i < 0 || i >= r.rot) continue;
    const bool up = r.interleaved ? i & 1 : i >= half;
    const int j = r.interleaved ? i >> 1 : up ? i - half : i;
    const int gap = r.interleaved ? 1 : half;
    y[n] = turned(y[n], x[up ? e + n - gap : e + n + gap], angles[2 * j], angles[2 * j + 1], up);
  }
  return make_float4(y[0], y[1], y[2], y[3]);
}

// One warp per token and `each` of its key/value heads, one after the other:
// their key rows and value rows, four elements a lane.
template <int kD, bool kFour>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int N = kD / 128;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= p.warps) return;
  const unsigned tok = w / p.groups, h0 = (w - tok * p.groups) * p.each;
  const unsigned s = tok / p.p.ntok, i = tok - s * p.p.ntok;
  const int64_t from = s * p.seq_ld + i * p.ld + h0 * kD + 4 * lane;
  const float *k = p.k + from, *v = p.x + from;
  float4 x[2][N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    x[0][n] = *reinterpret_cast<const float4 *>(k + 128 * n);
    x[1][n] = *reinterpret_cast<const float4 *>(v + 128 * n);
  }
  if (i >= tokens_of(p.p, s)) return;
  const int pos = seq_length(p.v, s) + i;
  const int page = seq_page(p.v, s, pos >> p.page_bits);
  if (page < 0) {
    if (lane == 0) record_error(p.err, DEVERR_NO_PAGE, s);
    return;
  }
  const float *angles = nullptr;
  if (p.r.table) {
    angles = angles_at(p.r, place_of(p.p, s, i));
    if (!angles && lane == 0) record_error(p.err, DEVERR_NO_ANGLE, s);
  }
  const bool lost = p.r.table && !angles;  // the keys' position has no angle
  uint8_t *row = page_row(p.v, p.layer, page, h0, 0, pos & (p.v.P - 1));
  Turn turn[N];
  if constexpr (kFour) {
#pragma unroll
    for (int n = 0; n < N; ++n) turn[n] = turn_of(p.r, 128 * n + 4 * lane, angles);
  }
  for (unsigned h = h0; h < h0 + p.each; ++h, k += kD, v += kD, row += p.v.head_bytes) {
    float4 next[2][N] = {};  // the next head's rows, while these are worked on
    if (h + 1 < h0 + p.each) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        next[0][n] = *reinterpret_cast<const float4 *>(k + kD + 128 * n);
        next[1][n] = *reinterpret_cast<const float4 *>(v + kD + 128 * n);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if constexpr (kFour) x[0][n] = turned4(turn[n], k + 128 * n, x[0][n]);
      else if (angles) x[0][n] = turned_any(p.r, k - 4 * lane, 128 * n + 4 * lane, angles, x[0][n]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint8_t *to = row + c * p.plane_bytes;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        __half d;
        const uint32_t word = quantize4(x[c][n], &d);
        // the factors of four blocks, joined in lane 0
        uint32_t f = c == 0 && lost ? 0x7fffu : __half_as_ushort(d);
        f |= __shfl_down_sync(0xffffffffu, f, 8) << 16;
        const uint32_t g = __shfl_down_sync(0xffffffffu, f, 16);
        if (lane == 0) *reinterpret_cast<uint2 *>(to + 8 * n) = make_uint2(f, g);
        *reinterpret_cast<uint32_t *>(to + kD / 16 + 128 * n + 4 * lane) = word;
        x[c][n] = next[c][n];
      }
    }
  }
}

__global__ void __launch_bounds__(kMaxSeq) advance_kernel(const __grid_constant__ PagesView v,
                                                          const int32_t *__restrict__ n) {
  pdl_launch_dependents();
  pdl_wait();
  const int s = threadIdx.x;
  if (s >= v.n_seq) return;
  const int len = seq_length(v, s), all = v.max_pages * v.P;
  v.length[s] = len + min(max(n[s], 0), all - len);
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" epq_status epq_pages_append(const epq_pages *pages, int layer, const float *k, const float *v, int ntok,
                                       const epq_append_opts *opts, epq_stream_t stream) {
  static const epq_append_opts kNone = {};
  const epq_append_opts &o = opts ? *opts : kNone;
  AppendParams p;
  epq_status st = pages_view(pages, &p.v);
  if (st != EPQ_OK) return st;
  if (!k || !v || layer < 0 || layer >= p.v.n_layers) return EPQ_ERR_ARG;
  if (ntok < 1 || static_cast<int64_t>(p.v.n_seq) * ntok * p.v.n_kv >= (1ll << 30) || (o.mask && !o.position && ntok > 64))
    return EPQ_ERR_SHAPE;
  st = rotation_view(o.rotation, p.v.D, &p.r);
  if (st != EPQ_OK) return st;
  p.ld = o.kv_ld ? o.kv_ld : static_cast<int64_t>(p.v.n_kv) * p.v.D;
  p.seq_ld = o.kv_seq_ld ? o.kv_seq_ld : ntok * p.ld;
  if (o.kv_ld < 0 || o.kv_seq_ld < 0) return EPQ_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || p.ld % 4 || p.seq_ld % 4 || !aligned_to(4, o.position, o.n_tok) ||
      !aligned_to(8, o.mask))
    return EPQ_ERR_ALIGN;
  p.p = {o.position, p.v.length, o.mask, o.n_tok, ntok};
  p.k = k, p.x = v, p.layer = layer;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  p.err = device_error_slot();
  if (!p.err) return EPQ_ERR_DEVICE;
  // what a token's heads share is worked out once for as many of them as leave
  // every SM 64 warps (8192 tokens x 8 heads: four to a warp 24.1 us, two 28.0,
  // when that was measured; 1551 x 16, a third of them used: two to a warp 5.6
  // us, four 6.8, eight 14.9)
  const int64_t tokens = static_cast<int64_t>(p.v.n_seq) * ntok;
  p.each = p.v.n_kv;
  while (p.each % 2 == 0 && tokens * (p.v.n_kv / p.each) < 64ll * dev.sm_count) p.each /= 2;
  p.groups = p.v.n_kv / p.each;
  p.warps = static_cast<unsigned>(tokens * p.groups);
  p.page_bits = p.v.P == 16 ? 4 : p.v.P == 32 ? 5 : p.v.P == 64 ? 6 : 7;
  p.plane_bytes = p.v.P * p.v.row;
  const bool four = rotates_by_four(p.r);
  void (*kernel)(AppendParams) = p.v.D == 128 ? (four ? append_kernel<128, true> : append_kernel<128, false>)
                                              : (four ? append_kernel<256, true> : append_kernel<256, false>);
  const cudaError_t e = launch_pdl(kernel, dim3((p.warps + kWarps - 1) / kWarps),
                                   dim3(32 * kWarps), 0, reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}

extern "C" epq_status epq_pages_advance(const epq_pages *pages, const int32_t *n, epq_stream_t stream) {
  PagesView v;
  const epq_status st = pages_view(pages, &v);
  if (st != EPQ_OK) return st;
  if (!n) return EPQ_ERR_ARG;
  if (!aligned_to(4, n)) return EPQ_ERR_ALIGN;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  const cudaError_t e =
      launch_pdl(advance_kernel, dim3(1), dim3(kMaxSeq), 0, reinterpret_cast<cudaStream_t>(stream), v, n);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
