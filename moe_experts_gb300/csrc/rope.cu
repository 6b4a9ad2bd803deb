// Rotary positions: frequencies, the table of cosines and sines, and the
// rotation of query and key heads (epq_rope_frequencies, epq_rope_table,
// epq_rope).
#include <algorithm>
#include <cmath>

#include "rope.cuh"

namespace epq {
namespace {

// ------------------------------------------------------------------ table
// One thread per (position, pair).  Angles in float64: at position 10^6 a
// float32 angle would be off by 0.03.  Run once per table, bound by the
// float64 cosine and sine.
__global__ void __launch_bounds__(256) table_kernel(const double *__restrict__ freq, int half, double magnitude,
                                                    int64_t n, float2 *__restrict__ table) {
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t x = blockIdx.x * 256ll + threadIdx.x; x < n; x += gridDim.x * 256ll) {
    const int64_t pos = x / half;
    double s, c;
    sincos(static_cast<double>(pos) * freq[x - pos * half], &s, &c);
    table[x] = make_float2(static_cast<float>(c * magnitude), static_cast<float>(s * magnitude));
  }
}

// ------------------------------------------------------------------ rotation
struct RopeParams {
  RotationView r;
  Places p;
  const float *x;
  float *y;
  int64_t x_ld, x_seq, y_ld, y_seq;
  int heads, dim;
  int pair_units, units, rows;  // units of a head (the pairs' first), heads that a CTA takes at a time
  unsigned *err;
};

template <int V>
struct Run;
template <>
struct Run<4> {
  using T = float4;
};
template <>
struct Run<1> {
  using T = float;
};

__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s) {
  const float y = turned(a, b, c, s, false);
  b = turned(b, a, c, s, true);
  a = y;
}

// A unit is what a thread reads of a head: V = 4: four pairs (half layout, two
// 16-byte reads) or two (interleaved, one); V = 1: one pair.  Units past the
// pairs are elements that are only copied, V at a time.
template <int V, bool kInter>
struct Unit {
  typename Run<V>::T a, b;
};

template <int V, bool kInter>
__device__ __forceinline__ void turn(Unit<V, kInter> &u, const float (&cs)[V == 4 && !kInter ? 8 : V == 4 ? 4 : 2]) {
  if constexpr (V == 1) {
    turn_pair(u.a, u.b, cs[0], cs[1]);
  } else if constexpr (kInter) {
    turn_pair(u.a.x, u.a.y, cs[0], cs[1]);
    turn_pair(u.a.z, u.a.w, cs[2], cs[3]);
  } else {
    turn_pair(u.a.x, u.b.x, cs[0], cs[1]);
    turn_pair(u.a.y, u.b.y, cs[2], cs[3]);
    turn_pair(u.a.z, u.b.z, cs[4], cs[5]);
    turn_pair(u.a.w, u.b.w, cs[6], cs[7]);
  }
}

// One CTA per token.  A thread keeps one unit, with its cosines and sines in
// registers, and goes through the heads with it, four of them on their way at a
// time.  Bound by DRAM: 40 heads of 128 of 4096 tokens, 169 MB, take 27.1 us (6.2
// TB/s, 0.92 of the copy rate); 8 tokens 2.4 us, one chain of position, angles,
// store.
template <int V, bool kInter>
__global__ void __launch_bounds__(1024) rope_kernel(const __grid_constant__ RopeParams p) {
  using T = typename Run<V>::T;
  constexpr int kAngles = V == 4 && !kInter ? 8 : V == 4 ? 4 : 2;
  constexpr bool kTwo = V == 1 || !kInter;  // a pair unit reads two places
  constexpr int kAhead = 4;
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x / p.p.ntok, i = blockIdx.x - s * p.p.ntok;
  const int u = threadIdx.x % p.units, h0 = threadIdx.x / p.units;
  const bool pairs = u < p.pair_units;
  int at, other = 0;  // the unit's first elements in a head
  if (pairs) {
    if constexpr (V == 4) {
      at = p.r.first + 4 * u;
      other = at + p.r.rot / 2;
    } else {
      at = p.r.first + (kInter ? 2 * u : u);
      other = kInter ? at + 1 : at + p.r.rot / 2;
    }
  } else {
    at = (u - p.pair_units) * V;
    if (at >= p.r.first) at += p.r.rot;
  }
  const float *x = p.x + s * p.x_seq + i * p.x_ld;
  float *y = p.y + s * p.y_seq + i * p.y_ld;
  const bool live = i < tokens_of(p.p, s);
  if (!live && p.x == p.y) return;
  bool turns = pairs && live;
  float cs[kAngles];
  if (turns) {
    const float *row = angles_at(p.r, place_of(p.p, s, i));
    if (!row) {
      record_error(p.err, DEVERR_NO_ANGLE, static_cast<unsigned>(blockIdx.x));
#pragma unroll
      for (int k = 0; k < kAngles; ++k) cs[k] = __int_as_float(0x7fffffff);
    } else if constexpr (V == 4) {
#pragma unroll
      for (int k = 0; k < kAngles; k += 4) {
        const float4 t = *reinterpret_cast<const float4 *>(row + kAngles * u + k);
        cs[k] = t.x, cs[k + 1] = t.y, cs[k + 2] = t.z, cs[k + 3] = t.w;
      }
    } else {
      const float2 t = *reinterpret_cast<const float2 *>(row + 2 * u);
      cs[0] = t.x, cs[1] = t.y;
    }
  }
  for (int h = h0; h < p.heads; h += kAhead * p.rows) {
    Unit<V, kInter> w[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int hk = h + k * p.rows;
      if (hk >= p.heads) break;
      w[k].a = *reinterpret_cast<const T *>(x + hk * p.dim + at);
      if (kTwo && pairs) w[k].b = *reinterpret_cast<const T *>(x + hk * p.dim + other);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int hk = h + k * p.rows;
      if (hk >= p.heads) break;
      if (turns) turn<V, kInter>(w[k], cs);
      *reinterpret_cast<T *>(y + hk * p.dim + at) = w[k].a;
      if (kTwo && pairs) *reinterpret_cast<T *>(y + hk * p.dim + other) = w[k].b;
    }
  }
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" epq_status epq_rope_frequencies(int rot_dim, double base, const epq_rope_scaling *scaling, double *freq,
                                           double *magnitude) {
  if (!freq || !magnitude || !std::isfinite(base) || !(base > 1.0)) return EPQ_ERR_ARG;
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > 1024) return EPQ_ERR_SHAPE;
  const int kind = scaling ? scaling->kind : EPQ_ROPE_PLAIN;
  if (kind < EPQ_ROPE_PLAIN || kind > EPQ_ROPE_BANDS) return EPQ_ERR_ARG;
  const double pi = 3.14159265358979323846;
  double factor = 1.0, context = 1.0, low = 1.0, high = 2.0;
  if (kind != EPQ_ROPE_PLAIN) {
    factor = scaling->factor;
    if (!std::isfinite(factor) || !(factor >= 1.0)) return EPQ_ERR_ARG;
  }
  if (kind == EPQ_ROPE_PARTS || kind == EPQ_ROPE_BANDS) {
    context = scaling->context, low = scaling->low, high = scaling->high;
    if (!std::isfinite(context) || !(context >= 1.0) || !(low > 0.0) || !(high > low) || !std::isfinite(high))
      return EPQ_ERR_ARG;
  }
  const auto pair_of = [&](double turns) {
    return rot_dim * std::log(context / (2.0 * pi * turns)) / (2.0 * std::log(base));
  };
  const double from = std::max(std::floor(pair_of(high)), 0.0);
  const double to = std::min(std::ceil(pair_of(low)), rot_dim - 1.0);
  for (int j = 0; j < rot_dim / 2; ++j) {
    const double f = std::pow(base, -2.0 * j / rot_dim);
    double slow = 0.0;  // how much of f / factor there is in the pair
    if (kind == EPQ_ROPE_LINEAR) slow = 1.0;
    if (kind == EPQ_ROPE_PARTS) slow = std::min(std::max((j - from) / std::max(to - from, 0.001), 0.0), 1.0);
    if (kind == EPQ_ROPE_BANDS)
      slow = 1.0 - std::min(std::max((context * f / (2.0 * pi) - low) / (high - low), 0.0), 1.0);
    freq[j] = f / factor * slow + f * (1.0 - slow);
  }
  *magnitude = kind == EPQ_ROPE_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return EPQ_OK;
}

extern "C" epq_status epq_rope_table(const double *freq, int rot_dim, double magnitude, int64_t n_pos, float *table,
                                     epq_stream_t stream) {
  if (!freq || !table || !std::isfinite(magnitude) || n_pos < 1) return EPQ_ERR_ARG;
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > 1024 || n_pos > (int64_t(1) << 30)) return EPQ_ERR_SHAPE;
  if (!aligned16(freq) || !aligned16(table)) return EPQ_ERR_ALIGN;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  const int64_t n = n_pos * (rot_dim / 2);
  const int grid = static_cast<int>(std::min<int64_t>((n + 255) / 256, 8ll * dev.sm_count));
  const cudaError_t e = launch_pdl(table_kernel, dim3(grid), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream),
                                   freq, rot_dim / 2, magnitude, n, reinterpret_cast<float2 *>(table));
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}

extern "C" epq_status epq_rope(const epq_rotation *rotation, const float *x, float *y, int n_seq, int ntok, int n_heads,
                               int head_dim, const epq_rope_opts *opts, epq_stream_t stream) {
  static const epq_rope_opts kNone = {};
  const epq_rope_opts &o = opts ? *opts : kNone;
  if (!rotation || !x || !y) return EPQ_ERR_ARG;
  if (n_seq < 1 || ntok < 1 || n_heads < 1 || n_heads > 65535 || head_dim < 2 || head_dim > 1024 ||
      static_cast<int64_t>(n_seq) * ntok > 0x7fffffffll || (o.mask && !o.position && ntok > 64))
    return EPQ_ERR_SHAPE;
  RopeParams p;
  const epq_status st = rotation_view(rotation, head_dim, &p.r);
  if (st != EPQ_OK) return st;
  const int64_t width = static_cast<int64_t>(n_heads) * head_dim;
  p.x = x, p.y = y;
  p.x_ld = o.x_ld ? o.x_ld : width;
  p.y_ld = o.y_ld ? o.y_ld : width;
  p.x_seq = o.x_seq_ld ? o.x_seq_ld : ntok * p.x_ld;
  p.y_seq = o.y_seq_ld ? o.y_seq_ld : ntok * p.y_ld;
  if ((ntok > 1 && p.y_ld < width) || (n_seq > 1 && p.y_seq < width) || o.x_ld < 0 || o.y_ld < 0 || o.x_seq_ld < 0 || o.y_seq_ld < 0 ||
      (x == y && (p.x_ld != p.y_ld || p.x_seq != p.y_seq)))
    return EPQ_ERR_ARG;
  if (!aligned_to(4, x, y, o.position, o.start, o.n_tok) || !aligned_to(8, o.mask)) return EPQ_ERR_ALIGN;
  p.p = {o.position, o.start, o.mask, o.n_tok, ntok};
  p.heads = n_heads, p.dim = head_dim;
  const bool four = aligned16(x) && aligned16(y) && head_dim % 4 == 0 && p.x_ld % 4 == 0 && p.y_ld % 4 == 0 &&
                    p.x_seq % 4 == 0 && p.y_seq % 4 == 0 && rotates_by_four(p.r);
  p.pair_units = !four ? p.r.rot / 2 : p.r.interleaved ? p.r.rot / 4 : p.r.rot / 8;
  p.units = p.pair_units + (x == y ? 0 : (head_dim - p.r.rot) / (four ? 4 : 1));
  p.rows = std::max(1, std::min(256 / p.units, n_heads));
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  p.err = device_error_slot();
  if (!p.err) return EPQ_ERR_DEVICE;
  void (*kernel)(RopeParams) = four ? (p.r.interleaved ? rope_kernel<4, true> : rope_kernel<4, false>)
                                    : (p.r.interleaved ? rope_kernel<1, true> : rope_kernel<1, false>);
  const cudaError_t e = launch_pdl(kernel, dim3(n_seq * ntok), dim3(p.units * p.rows), 0,
                                   reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
