// Biases, penalties for repeated tokens and grammar masks on the logits of
// drafted tokens (epq_logits_adjust).
//
//   l += b(v);  seen: l = l > 0 ? l / r : l r;  n > 0: l -= f n + p;  not allowed: -inf
//
// n(v) counts the row's generated tokens v: the history behind the prompt, and
// the drafted tokens on the row's path.  A CTA takes kChunk tokens of the
// vocabulary for some rows of one sequence.  It goes through the history and
// the biases once and keeps, for each of its tokens, the count, whether the
// prompt has it, and the last bias entry that names it in shared memory; only
// the path differs between the rows, and is added and taken away again.
// Integer counts and a maximum of indices do not depend on the order in which
// threads come, so the result does not either.
#include <algorithm>

#include "common.cuh"

namespace epq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;  // tokens of a CTA: 16 a thread
constexpr int kMaxTokens = 64;

struct LogitsParams {
  const float *x;
  float *y;
  int64_t ld, out_ld;
  int vocab, ntok;
  int rows_per_cta, row_groups;
  const float *penalties;
  const int32_t *history, *history_len, *prompt_len;
  int max_history;
  const int32_t *tokens;
  const uint64_t *mask;
  const int32_t *n_tok;
  const int32_t *bias_ids;
  const float *bias;
  int n_bias;
  const uint32_t *allowed;
  int words;  // of a row of `allowed`
};

// What a CTA knows of its tokens.  A token's note: its count, and in the top
// bit whether the prompt has it.
constexpr uint32_t kRead = 0x80000000u;

__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ LogitsParams p) {
  __shared__ uint32_t note[kChunk];
  __shared__ int entry[kChunk];  // 1 + the last bias entry, 0: none
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  const int s = blockIdx.x / p.row_groups, r0 = (blockIdx.x - s * p.row_groups) * p.rows_per_cta;
  const int v0 = blockIdx.y * kChunk, nv = min(kChunk, p.vocab - v0);
  const int live = p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok;
  const int r1 = min(r0 + p.rows_per_cta, p.ntok);
  const float rep = p.penalties ? p.penalties[3 * s] : 1.0f;
  const float freq = p.penalties ? p.penalties[3 * s + 1] : 0.0f, pres = p.penalties ? p.penalties[3 * s + 2] : 0.0f;
  if (r0 < live) {
    for (int i = tid; i < kChunk; i += kThreads) note[i] = 0, entry[i] = 0;
    __syncthreads();
    if (p.history) {
      const int n = p.history_len ? min(max(p.history_len[s], 0), p.max_history) : p.max_history;
      const int given = p.prompt_len ? min(max(p.prompt_len[s], 0), n) : 0;
      const int32_t *h = p.history + static_cast<int64_t>(s) * p.max_history;
      for (int i = tid; i < n; i += kThreads) {
        const unsigned at = static_cast<unsigned>(h[i]) - v0;
        if (at >= static_cast<unsigned>(nv)) continue;
        if (i < given) atomicOr(&note[at], kRead);
        else atomicAdd(&note[at], 1u);
      }
    }
    for (int i = tid; i < p.n_bias; i += kThreads) {
      const unsigned at = static_cast<unsigned>(p.bias_ids[static_cast<int64_t>(s) * p.n_bias + i]) - v0;
      if (at < static_cast<unsigned>(nv)) atomicMax(&entry[at], i + 1);
    }
    __syncthreads();
  }
  for (int r = r0; r < r1; ++r) {
    const int64_t row = static_cast<int64_t>(s) * p.ntok + r;
    const float *x = p.x + row * p.ld + v0;
    float *y = p.y + row * p.out_ld + v0;
    if (r >= live) {
      if (p.x != p.y)
        for (int i = tid; i < nv; i += kThreads) y[i] = x[i];
      continue;
    }
    // the drafted tokens on the row's path, one a thread
    unsigned mine = 0xffffffffu;
    if (p.tokens && tid < live) {
      const uint64_t path = p.mask ? p.mask[row] : ~0ull >> (63 - r);
      if (path >> tid & 1) mine = static_cast<unsigned>(p.tokens[static_cast<int64_t>(s) * p.ntok + tid]) - v0;
      if (mine >= static_cast<unsigned>(nv)) mine = 0xffffffffu;
      if (mine != 0xffffffffu) atomicAdd(&note[mine], 1u);
    }
    __syncthreads();
    const uint32_t *allowed = p.allowed ? p.allowed + row * p.words + v0 / 32 : nullptr;
    for (int i = tid; i < nv; i += kThreads) {
      float l = x[i];
      const int e = entry[i];
      if (e) l = __fadd_rn(l, p.bias[static_cast<int64_t>(s) * p.n_bias + e - 1]);
      const uint32_t w = note[i];
      if (w) {
        l = l > 0.0f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
        const uint32_t n = w & ~kRead;
        if (n) l = __fsub_rn(l, __fadd_rn(__fmul_rn(freq, static_cast<float>(n)), pres));
      }
      if (allowed && !(allowed[i >> 5] >> (i & 31) & 1)) l = -INFINITY;
      y[i] = l;
    }
    __syncthreads();
    if (mine != 0xffffffffu) atomicSub(&note[mine], 1u);
  }
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" epq_status epq_logits_adjust(const float *logits, int64_t vocab, int n_seq, int ntok,
                                        const epq_logits_opts *opts, float *out, epq_stream_t stream) {
  static const epq_logits_opts kNone = {};
  const epq_logits_opts &o = opts ? *opts : kNone;
  if (!logits || !out) return EPQ_ERR_ARG;
  if (vocab < 1 || vocab > (1 << 24) || n_seq < 1 || ntok < 1 || static_cast<int64_t>(n_seq) * ntok >= (1 << 24) ||
      (o.tokens && ntok > kMaxTokens) || o.max_history < 0 || o.max_history > (1 << 24) || o.n_bias < 0 ||
      o.n_bias > (1 << 24))
    return EPQ_ERR_SHAPE;
  if ((o.max_history > 0 && !o.history) || (o.n_bias > 0 && (!o.bias_ids || !o.bias)) || (o.ld && o.ld < vocab) ||
      (o.out_ld && o.out_ld < vocab))
    return EPQ_ERR_ARG;
  LogitsParams p = {};
  p.x = logits, p.y = out;
  p.ld = o.ld ? o.ld : vocab;
  p.out_ld = o.out_ld ? o.out_ld : vocab;
  if (logits == out && p.ld != p.out_ld) return EPQ_ERR_ARG;
  if (!aligned_to(4, logits, out, o.penalties, o.history, o.history_len, o.prompt_len, o.tokens, o.n_tok, o.bias_ids,
                  o.bias, o.allowed) || !aligned_to(8, o.mask))
    return EPQ_ERR_ALIGN;
  p.vocab = static_cast<int>(vocab), p.ntok = ntok;
  p.penalties = o.penalties;
  p.history = o.max_history ? o.history : nullptr;
  p.history_len = o.history_len, p.prompt_len = o.prompt_len, p.max_history = o.max_history;
  p.tokens = o.tokens, p.mask = o.mask, p.n_tok = o.n_tok;
  p.bias_ids = o.bias_ids, p.bias = o.bias, p.n_bias = o.n_bias;
  p.allowed = o.allowed, p.words = static_cast<int>((vocab + 31) / 32);
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  const int chunks = (p.vocab + kChunk - 1) / kChunk;
  // rows share the pass over the history; but all SMs have CTAs
  const int64_t want = std::max<int64_t>(1, 4ll * dev.sm_count / chunks);  // CTAs of a chunk
  const int groups = static_cast<int>(std::min<int64_t>(ntok, std::max<int64_t>(1, want / n_seq)));
  p.rows_per_cta = (ntok + groups - 1) / groups;
  p.row_groups = (ntok + p.rows_per_cta - 1) / p.rows_per_cta;
  const cudaError_t e = launch_pdl(adjust_kernel, dim3(n_seq * p.row_groups, chunks), dim3(kThreads), 0,
                                   reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
