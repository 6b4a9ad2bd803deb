// Any number of new rows brought into a paged Q8_0 cache, the keys rotated on
// the way (epq_pages_append), and their commit (epq_pages_advance).
//
//   row = (d_b, c_e):  d_b = fp16(max_e |x_e| / 127),  c_e = rint(x_e / d_b)
//
// over blocks b of 32 elements, x the value, or the key after its rotation.
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
  int64_t rows;  // sequences * tokens * heads
  unsigned *err;
};

// The rotation of elements e .. e + 3 of a head's row `x` (`a` holds them).
// kFour: pairs, cosines and sines lie in 16-byte words.
template <bool kFour>
__device__ __forceinline__ void rotate4(const RotationView &r, const float *x, int e, const float *angles, float4 &a) {
  const int at = e - r.first, half = r.rot / 2;
  if constexpr (kFour) {
    if (at < 0 || at >= r.rot) return;
    if (r.interleaved) {
      const float4 t = *reinterpret_cast<const float4 *>(angles + at);
      a = make_float4(turned(a.x, a.y, t.x, t.y, false), turned(a.y, a.x, t.x, t.y, true),
                      turned(a.z, a.w, t.z, t.w, false), turned(a.w, a.z, t.z, t.w, true));
    } else {
      const bool up = at >= half;
      const float4 b = *reinterpret_cast<const float4 *>(x + (up ? e - half : e + half));
      const float *cs = angles + 2 * (up ? at - half : at);
      const float4 t = *reinterpret_cast<const float4 *>(cs), w = *reinterpret_cast<const float4 *>(cs + 4);
      a = make_float4(turned(a.x, b.x, t.x, t.y, up), turned(a.y, b.y, t.z, t.w, up), turned(a.z, b.z, w.x, w.y, up),
                      turned(a.w, b.w, w.z, w.w, up));
    }
  } else {
    float y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int i = at + n;
      if (i < 0 || i >= r.rot) continue;
      const bool up = r.interleaved ? i & 1 : i >= half;
      const int j = r.interleaved ? i >> 1 : up ? i - half : i;
      const int gap = r.interleaved ? 1 : half;
      y[n] = turned(y[n], x[up ? e + n - gap : e + n + gap], angles[2 * j], angles[2 * j + 1], up);
    }
    a = make_float4(y[0], y[1], y[2], y[3]);
  }
}

// One warp per (token, key/value head): its key row and its value row, four
// elements a lane.
template <int kD, bool kFour>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int N = kD / 128;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= p.rows) return;
  const int head = static_cast<int>(w % p.v.n_kv), tok = static_cast<int>(w / p.v.n_kv);
  const int s = tok / p.p.ntok, i = tok - s * p.p.ntok;
  const int64_t from = s * p.seq_ld + i * p.ld + head * kD;
  float4 x[2][N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    x[0][n] = *reinterpret_cast<const float4 *>(p.k + from + 128 * n + 4 * lane);
    x[1][n] = *reinterpret_cast<const float4 *>(p.x + from + 128 * n + 4 * lane);
  }
  if (i >= tokens_of(p.p, s)) return;
  const int pos = seq_length(p.v, s) + i;
  const int page = seq_page(p.v, s, pos / p.v.P);
  if (page < 0) {
    if (lane == 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(s));
    return;
  }
  bool lost = false;  // the key's position has no angle
  if (p.r.table) {
    const float *angles = angles_at(p.r, place_of(p.p, s, i));
    lost = angles == nullptr;
    if (!lost) {
#pragma unroll
      for (int n = 0; n < N; ++n) rotate4<kFour>(p.r, p.k + from, 128 * n + 4 * lane, angles, x[0][n]);
    } else if (lane == 0) {
      record_error(p.err, DEVERR_NO_ANGLE, static_cast<unsigned>(s));
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint8_t *row = page_row(p.v, p.layer, page, head, c, pos % p.v.P);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      __half d;
      const uint32_t word = quantize4(x[c][n], &d);
      // the factors of four blocks, joined in lane 0
      uint32_t f = __half_as_ushort(d);
      if (c == 0 && lost) f = 0x7fffu;
      f |= __shfl_down_sync(0xffffffffu, f, 8) << 16;
      const uint32_t g = __shfl_down_sync(0xffffffffu, f, 16);
      if (lane == 0) *reinterpret_cast<uint2 *>(row + 8 * n) = make_uint2(f, g);
      *reinterpret_cast<uint32_t *>(row + kD / 16 + 128 * n + 4 * lane) = word;
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
  p.rows = static_cast<int64_t>(p.v.n_seq) * ntok * p.v.n_kv;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  p.err = device_error_slot();
  if (!p.err) return EPQ_ERR_DEVICE;
  const bool four = rotates_by_four(p.r);
  void (*kernel)(AppendParams) = p.v.D == 128 ? (four ? append_kernel<128, true> : append_kernel<128, false>)
                                              : (four ? append_kernel<256, true> : append_kernel<256, false>);
  const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>((p.rows + kWarps - 1) / kWarps)),
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
