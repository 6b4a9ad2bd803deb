// Causal attention of a prompt's appended rows over a paged Q8_0 cache
// (epq_attention_prompt).
//
//   s_ij = scale q_i . k_j,  o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// over the positions j <= length + i.  The rows of one (sequence, key/value
// head) are its tokens times its `group` query heads (row r: token r / group,
// head r % group).  One pass over the positions in tiles of 32, dequantized
// into shared memory, with a running maximum and sum per row; a warp has two
// rows, a lane a position of the scores and D/32 columns of the output.
#include <algorithm>
#include <cmath>

#include "pages.cuh"

namespace epq {
namespace {

constexpr int kTile = 32, kWarps = 8, kWarpRows = 2, kRows = kWarps * kWarpRows;

struct PromptParams {
  PagesView v;
  const float *q;
  const int32_t *n_tok;
  int64_t q_ld, q_seq_ld;
  int layer, n_heads, group, ntok, window, tiles;
  float scale;
  float *out;
  unsigned *err;
};

template <int kD>
__global__ void __launch_bounds__(32 * kWarps) prompt_kernel(const __grid_constant__ PromptParams p) {
  constexpr int kLd = kD + 4;
  extern __shared__ __align__(16) float smem[];
  float *ks = smem, *vs = ks + kTile * kLd, *qs = vs + kTile * kLd;  // qs [kRows][kD]
  __shared__ float lost[kTile];  // NaN: a factor of the position is not finite; -inf: it has no page
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x % p.tiles, sh = blockIdx.x / p.tiles;
  const int h = sh % p.v.n_kv, s = sh / p.v.n_kv;
  const int n = p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok;
  const int len = seq_length(p.v, s);
  const int r0 = tile * kRows, rows = n * p.group;
  const auto out_row = [&](int r) {
    return p.out + (static_cast<int64_t>(s) * p.ntok + r / p.group) * p.n_heads * kD + (h * p.group + r % p.group) * kD;
  };
  for (int x = tid; x < kRows * kD; x += 32 * kWarps) {
    const int r = r0 + x / kD, e = x % kD;
    qs[x] = r < rows ? p.q[s * p.q_seq_ld + (r / p.group) * p.q_ld + (h * p.group + r % p.group) * kD + e] * p.scale : 0.0f;
    if (r >= rows && r < p.ntok * p.group) out_row(r)[e] = 0.0f;
  }
  if (r0 >= rows) return;
  const int t0 = r0 / p.group, t1 = (min(r0 + kRows, rows) - 1) / p.group;
  const int begin = p.window ? max(0, len + t0 - p.window + 1) : 0, end = len + t1 + 1;
  float top[kWarpRows], den[kWarpRows], o[kWarpRows][kD / 32];
#pragma unroll
  for (int k = 0; k < kWarpRows; ++k) {
    top[k] = -INFINITY, den[k] = 0.0f;
#pragma unroll
    for (int e = 0; e < kD / 32; ++e) o[k][e] = 0.0f;
  }
  for (int j0 = begin; j0 < end; j0 += kTile) {
    __syncthreads();
    for (int j = warp; j < kTile; j += kWarps) {
      const int pos = j0 + j;
      const int page = pos < end ? seq_page(p.v, s, pos / p.v.P) : -1;
      const uint8_t *kr = page >= 0 ? page_row(p.v, p.layer, page, h, 0, pos % p.v.P) : nullptr;
      const uint8_t *vr = page >= 0 ? page_row(p.v, p.layer, page, h, 1, pos % p.v.P) : nullptr;
      if (!kr && pos < end && lane == 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(s));
      bool bad = false;
#pragma unroll
      for (int e = 0; e < kD / 32; ++e) {
        float a = 0.0f, b = 0.0f;
        if (kr) {
          const float fk = __half2float(reinterpret_cast<const __half *>(kr)[e]);
          const float fv = __half2float(reinterpret_cast<const __half *>(vr)[e]);
          bad |= !isfinite(fk) || !isfinite(fv);
          a = isfinite(fk) ? fk * reinterpret_cast<const int8_t *>(kr + kD / 16)[32 * e + lane] : 0.0f;
          b = isfinite(fv) ? fv * reinterpret_cast<const int8_t *>(vr + kD / 16)[32 * e + lane] : 0.0f;
        }
        ks[j * kLd + 32 * e + lane] = a;
        vs[j * kLd + 32 * e + lane] = b;
      }
      if (lane == 0) lost[j] = !kr ? -INFINITY : bad ? __int_as_float(0x7fffffff) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarpRows; ++k) {
      const int row = warp * kWarpRows + k, at = len + (r0 + row) / p.group, pos = j0 + lane;
      const bool sees = r0 + row < rows && pos <= at && (!p.window || pos > at - p.window);
      float sc = 0.0f;
      for (int e = 0; e < kD; e += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(qs + row * kD + e);
        const float4 b = *reinterpret_cast<const float4 *>(ks + lane * kLd + e);
        sc = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, sc))));
      }
      sc = sees ? sc + lost[lane] : -INFINITY;
      const bool nan = __any_sync(0xffffffffu, isnan(sc));
      const float up = nan ? __int_as_float(0x7fffffff) : fmaxf(top[k], warp_max_all(sc));
      const float ref = up == -INFINITY ? 0.0f : up;
      const float keep = expf(top[k] - ref), w = expf(sc - ref);
      top[k] = isnan(top[k]) ? top[k] : up;
      den[k] = den[k] * keep + warp_sum_xor<32>(w);
#pragma unroll
      for (int e = 0; e < kD / 32; ++e) o[k][e] *= keep;
      for (int j = 0; j < kTile; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
        for (int e = 0; e < kD / 32; ++e) o[k][e] = fmaf(wj, vs[j * kLd + 32 * e + lane], o[k][e]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kWarpRows; ++k) {
    const int r = r0 + warp * kWarpRows + k;
    if (r >= rows) continue;
#pragma unroll
    for (int e = 0; e < kD / 32; ++e) out_row(r)[32 * e + lane] = den[k] != 0.0f ? o[k][e] / den[k] : 0.0f;
  }
}

bool sizes_ok(const epq_pages *pages, int n_heads, int ntok) {
  return pages_sizes_ok(pages) && n_heads >= 1 && n_heads % pages->n_kv_heads == 0 && n_heads / pages->n_kv_heads <= 16 &&
         ntok >= 1 && static_cast<int64_t>(pages->n_seq) * ntok < (1 << 24);
}

LaunchOnce g_launch[2];

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" size_t epq_attention_prompt_workspace_bytes(const epq_pages *pages, int n_heads, int ntok) {
  return sizes_ok(pages, n_heads, ntok) ? 16 : 0;
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
  p.q = q, p.n_tok = o.n_tok, p.layer = layer, p.n_heads = n_heads, p.group = n_heads / p.v.n_kv, p.ntok = ntok;
  p.window = o.window, p.scale = scale, p.out = out;
  p.tiles = (ntok * p.group + kRows - 1) / kRows;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  p.err = device_error_slot();
  if (!p.err) return EPQ_ERR_DEVICE;
  void (*kernel)(PromptParams) = p.v.D == 128 ? prompt_kernel<128> : prompt_kernel<256>;
  const size_t smem = 4 * (2 * kTile * (p.v.D + 4) + kRows * p.v.D);
  cudaError_t e = g_launch[p.v.D == 256].prepare(dev.device, kernel, 32 * kWarps, smem, false, nullptr);
  if (e == cudaSuccess)
    e = launch_pdl(kernel, dim3(static_cast<unsigned>(p.tiles * p.v.n_kv * p.v.n_seq)), dim3(32 * kWarps), smem,
                   reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
