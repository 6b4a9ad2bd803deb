// Attention of drafted tokens over a paged Q8_0 cache (epq_attention_tree).
//
//   s_ij = scale q_i . k_j,  o_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// over the committed positions and the drafted tokens that token i's mask
// names.  Two launches: append_kernel quantizes the new rows into their pages,
// tree_kernel (one CTA per sequence, token and query head) makes one pass over
// the positions with a running maximum and sum per warp and joins the warps.
#include <cmath>

#include "pages.cuh"

namespace epq {
namespace {

constexpr int kMaxGroupTree = 16;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct TreeParams {
  PagesView v;
  const float *q, *k_new, *v_new;
  const uint64_t *mask;
  const int32_t *n_tok;
  int64_t q_ld, q_seq_ld, kv_ld, kv_seq_ld;
  int layer, n_heads, group, ntok;
  float scale;
  float *out;
  unsigned *err;
};

__device__ __forceinline__ int tree_size(const TreeParams &p, int s) {
  return p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok;
}

__device__ __forceinline__ uint64_t token_mask(const TreeParams &p, int s, int i, int n) {
  const uint64_t m = p.mask ? p.mask[s * p.ntok + i] : ~0ull >> (63 - i);
  return n >= 64 ? m : m & ((1ull << n) - 1);
}

// Q8_0 of one 32-element run held one element per lane (the packer's
// arithmetic: factor fp16(max|x| / 127), codes rint(x / factor) clamped to
// +-127, zero codes for a zero factor).
__device__ __forceinline__ void q8_block(float x, uint16_t *d_out, int8_t *q_out) {
  x = __fadd_rn(x, 0.0f);  // -0 -> +0
  float a = fabsf(x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  const __half dh = __float2half_rn(__fdiv_rn(a, 127.0f));
  const float d = __half2float(dh);
  float q = 0.0f;
  if (d != 0.0f) q = fminf(fmaxf(rintf(__fdiv_rn(x, d)), -127.0f), 127.0f);
  *q_out = static_cast<int8_t>(q);
  *d_out = __half_as_ushort(dh);
}

// Grid (n_kv, ntok, n_seq): one new key row and one value row.
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ TreeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, i = blockIdx.y, s = blockIdx.z;
  if (i >= tree_size(p, s)) return;
  const int pos = seq_length(p.v, s) + i;
  const int page = seq_page(p.v, s, pos / p.v.P);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (page < 0) {
    if (threadIdx.x == 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(s));
    return;
  }
  const int nblk = p.v.D / 32;
  for (int b = warp; b < 2 * nblk; b += kWarps) {
    const int c = b / nblk, bb = b % nblk;
    const float x = (c ? p.v_new : p.k_new)[s * p.kv_seq_ld + i * p.kv_ld + h * p.v.D + 32 * bb + lane];
    uint8_t *row = page_row(p.v, p.layer, page, h, c, pos % p.v.P);
    uint16_t d;
    int8_t q;
    q8_block(x, &d, &q);
    row[2 * nblk + 32 * bb + lane] = static_cast<uint8_t>(q);
    if (lane == 0) *reinterpret_cast<uint16_t *>(row + 2 * bb) = d;
  }
}

// Grid (n_heads, ntok, n_seq).  Lane l of a warp holds elements 4l .. 4l+3 of
// each 128-element chunk.
template <int NCH>
__global__ void __launch_bounds__(kThreads) tree_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float part[kWarps][NCH * 128 + 2];
  pdl_launch_dependents();
  pdl_wait();
  const int hq = blockIdx.x, i = blockIdx.y, s = blockIdx.z;
  const int h = hq / p.group, D = NCH * 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = tree_size(p, s);
  float *out = p.out + (static_cast<int64_t>(s) * p.ntok + i) * p.n_heads * D + hq * D;
  if (i >= n) {
    for (int e = threadIdx.x; e < D; e += kThreads) out[e] = 0.0f;
    return;
  }
  const int len = seq_length(p.v, s);
  const uint64_t mask = token_mask(p, s, i, n);
  float4 q[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
    q[c] = *reinterpret_cast<const float4 *>(p.q + s * p.q_seq_ld + i * p.q_ld + hq * D + 128 * c + 4 * lane);
  float m = -INFINITY, z = 0.0f;
  float4 o[NCH] = {};
  for (int pos = warp; pos < len + n; pos += kWarps) {
    if (pos >= len && !(mask >> (pos - len) & 1)) continue;
    const int page = seq_page(p.v, s, pos / p.v.P);
    if (page < 0) {
      if (lane == 0) record_error(p.err, DEVERR_NO_PAGE, static_cast<unsigned>(s));
      continue;
    }
    float dot = 0.0f;
    const uint8_t *kr = page_row(p.v, p.layer, page, h, 0, pos % p.v.P);
    const uint8_t *vr = page_row(p.v, p.layer, page, h, 1, pos % p.v.P);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int e = 128 * c + 4 * lane;
      const float d = __half2float(*reinterpret_cast<const __half *>(kr + 2 * (e / 32)));
      const char4 k = *reinterpret_cast<const char4 *>(kr + D / 16 + e);
      dot = fmaf(d, fmaf(k.x, q[c].x, fmaf(k.y, q[c].y, fmaf(k.z, q[c].z, k.w * q[c].w))), dot);
    }
    const float sc = warp_sum_xor<32>(dot) * p.scale;
    const float m2 = fmaxf(m, sc);
    const float keep = m == m2 ? 1.0f : expf(m - m2), w = expf(sc - m2);
    m = m2;
    z = fmaf(z, keep, w);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int e = 128 * c + 4 * lane;
      const float d = __half2float(*reinterpret_cast<const __half *>(vr + 2 * (e / 32))) * w;
      const char4 x = *reinterpret_cast<const char4 *>(vr + D / 16 + e);
      o[c].x = fmaf(o[c].x, keep, d * x.x);
      o[c].y = fmaf(o[c].y, keep, d * x.y);
      o[c].z = fmaf(o[c].z, keep, d * x.z);
      o[c].w = fmaf(o[c].w, keep, d * x.w);
    }
  }
  if (lane == 0) part[warp][D] = m, part[warp][D + 1] = z;
#pragma unroll
  for (int c = 0; c < NCH; ++c) *reinterpret_cast<float2 *>(&part[warp][128 * c + 4 * lane]) = make_float2(o[c].x, o[c].y),
    *reinterpret_cast<float2 *>(&part[warp][128 * c + 4 * lane + 2]) = make_float2(o[c].z, o[c].w);
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][D]);
  float sum = 0.0f, f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = part[w][D + 1] > 0.0f || part[w][D + 1] != part[w][D + 1] ? expf(part[w][D] - top) : 0.0f;
    sum = fmaf(f[w], part[w][D + 1], sum);
  }
  for (int e = threadIdx.x; e < D; e += kThreads) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w)
      if (f[w] != 0.0f) x = fmaf(f[w], part[w][e], x);
    out[e] = sum != 0.0f ? x / sum : 0.0f;
  }
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" size_t epq_attention_tree_workspace_bytes(const epq_pages *pages, int n_heads, int ntok) {
  if (!pages_sizes_ok(pages) || n_heads < 1 || n_heads % pages->n_kv_heads ||
      n_heads / pages->n_kv_heads > kMaxGroupTree || ntok < 1 || ntok > kMaxTree)
    return 0;
  return 16;
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
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(append_kernel, dim3(n_kv, ntok, p.v.n_seq), dim3(kThreads), 0, s, p);
  const dim3 grid(n_heads, ntok, p.v.n_seq);
  if (e == cudaSuccess)
    e = D == 128 ? launch_pdl(tree_kernel<1>, grid, dim3(kThreads), 0, s, p)
                 : launch_pdl(tree_kernel<2>, grid, dim3(kThreads), 0, s, p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
