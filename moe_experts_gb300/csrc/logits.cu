// Biases, penalties for repeated tokens and grammar masks on the logits of
// drafted tokens (epq_logits_adjust).
//
//   l += b(v);  seen: l = l > 0 ? l / r : l r;  n > 0: l -= f n + p;  not allowed: -inf
//
// n(v) counts the row's generated tokens v: the history behind the prompt, and
// the drafted tokens on the row's path.  A CTA takes kChunk tokens of the
// vocabulary for some rows of one sequence.  It goes through the history and
// the biases once and keeps a note for each of its tokens in shared memory; only
// the path differs between the rows, and the thread that owns a drafted token
// adds it to its note for the row and takes it away again, so the rows need no
// barrier.  Integer counts and a maximum of indices do not depend on the order
// in which threads come, so the result does not either.
#include <algorithm>

#include "common.cuh"

namespace epq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 2048;  // tokens of a CTA: 8 a thread
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

// A token's note: its count, whether the prompt has it, whether it has a bias.
// Most are 0: the token's logit changes by the mask alone.
constexpr uint32_t kRead = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3fffffffu;

__device__ __forceinline__ float adjusted(float l, uint32_t w, float bias, const float (&pen)[3]) {
  if (w & kBiased) l = __fadd_rn(l, bias);
  if (w & ~kBiased) l = l > 0.0f ? __fdiv_rn(l, pen[0]) : __fmul_rn(l, pen[0]);
  if (w & kCount) l = __fsub_rn(l, __fadd_rn(__fmul_rn(pen[1], static_cast<float>(w & kCount)), pen[2]));
  return l;
}

// kFour: a thread has four tokens next to one another, in 16-byte words (rows
// that begin at 16 bytes); else every 256th.
template <bool kFour>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ LogitsParams p) {
  constexpr int kEach = kChunk / kThreads;
  __shared__ __align__(16) uint32_t note[kChunk];
  __shared__ __align__(16) float added[kChunk];  // first 1 + the last bias entry (0: none), then that bias
  __shared__ int drafted[kMaxTokens];            // the drafted tokens' places in the chunk, or -1
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  const int s = blockIdx.x / p.row_groups, r0 = (blockIdx.x - s * p.row_groups) * p.rows_per_cta;
  const int v0 = blockIdx.y * kChunk, nv = min(kChunk, p.vocab - v0);
  const int r1 = min(r0 + p.rows_per_cta, p.ntok);
  const auto place = [&](int k) { return kFour ? 4 * (tid + kThreads * (k / 4)) + k % 4 : tid + kThreads * k; };
  const auto load = [&](int r, float (&x)[kEach]) {
    const float *row = p.x + (static_cast<int64_t>(s) * p.ntok + r) * p.ld + v0;
    if constexpr (kFour) {
#pragma unroll
      for (int k = 0; k < kEach; k += 4)
        if (place(k) < nv) *reinterpret_cast<float4 *>(x + k) = *reinterpret_cast<const float4 *>(row + place(k));
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (place(k) < nv) x[k] = row[place(k)];
    }
  };
  __align__(16) float x[kEach], ahead[kEach];  // a row, and the next one while the row is worked on
  load(r0, ahead);
  const int live = p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok;
  float pen[3] = {1.0f, 0.0f, 0.0f};
  if (p.penalties) {
#pragma unroll
    for (int k = 0; k < 3; ++k) pen[k] = p.penalties[3 * s + k];
  }
  uint64_t mine = 0;  // the drafted tokens that this thread has
  if (r0 < live) {
    int *entry = reinterpret_cast<int *>(added);
    for (int i = 4 * tid; i < kChunk; i += 4 * kThreads) {
      *reinterpret_cast<uint4 *>(note + i) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4 *>(entry + i) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (p.history) {
      const int n = p.history_len ? min(max(p.history_len[s], 0), p.max_history) : p.max_history;
      const int given = p.prompt_len ? min(max(p.prompt_len[s], 0), n) : 0;
      const int32_t *h = p.history + static_cast<int64_t>(s) * p.max_history;
#pragma unroll 8
      for (int i = tid; i < n; i += kThreads) {
        const unsigned at = static_cast<unsigned>(h[i]) - v0;
        if (at >= static_cast<unsigned>(nv)) continue;
        if (i < given) atomicOr(&note[at], kRead);
        else atomicAdd(&note[at], 1u);
      }
    }
    for (int i = tid; i < p.n_bias; i += kThreads) {
      const unsigned at = static_cast<unsigned>(p.bias_ids[static_cast<int64_t>(s) * p.n_bias + i]) - v0;
      if (at >= static_cast<unsigned>(nv)) continue;
      atomicOr(&note[at], kBiased);
      atomicMax(&entry[at], i + 1);
    }
    if (tid < kMaxTokens) {
      unsigned at = 0xffffffffu;
      if (p.tokens && tid < live) at = static_cast<unsigned>(p.tokens[static_cast<int64_t>(s) * p.ntok + tid]) - v0;
      drafted[tid] = at < static_cast<unsigned>(nv) ? static_cast<int>(at) : -1;
    }
    __syncthreads();
    if (p.n_bias) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int e = entry[place(k)];
        if (e) added[place(k)] = p.bias[static_cast<int64_t>(s) * p.n_bias + e - 1];
      }
    }
    if (p.tokens) {
#pragma unroll 8
      for (int j = 0; j < kMaxTokens; ++j) {
        const int at = drafted[j];
        if (at >= 0 && (kFour ? at / 4 : at) % kThreads == tid) mine |= 1ull << j;
      }
    }
  }
  for (int r = r0; r < r1; ++r) {
    const int64_t row = static_cast<int64_t>(s) * p.ntok + r;
    float *y = p.y + row * p.out_ld + v0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) x[k] = ahead[k];
    if (r + 1 < r1) load(r + 1, ahead);
    if (r < live) {
      uint64_t path = 0;
      if (mine) {
        path = mine & (p.mask ? p.mask[row] : ~0ull >> (63 - r));
        for (uint64_t b = path; b; b &= b - 1) ++note[drafted[__ffsll(b) - 1]];
      }
      const uint32_t *allowed = p.allowed ? p.allowed + row * p.words + v0 / 32 : nullptr;
#pragma unroll
      for (int k = 0; k < kEach; k += 4) {
        uint32_t w[4], in[4];
        if constexpr (kFour) {
          *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(note + place(k));
          const uint32_t bits = allowed && place(k) < nv ? allowed[place(k) >> 5] >> (place(k) & 31) : ~0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) in[i] = bits >> i & 1;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = place(k + i);
            w[i] = note[at];
            in[i] = allowed && at < nv ? allowed[at >> 5] >> (at & 31) & 1 : 1;
          }
        }
        if (w[0] | w[1] | w[2] | w[3]) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (w[i]) x[k + i] = adjusted(x[k + i], w[i], added[place(k + i)], pen);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!in[i]) x[k + i] = -INFINITY;
      }
      for (uint64_t b = path; b; b &= b - 1) --note[drafted[__ffsll(b) - 1]];
    } else if (p.x == p.y) {
      continue;
    }
    if constexpr (kFour) {
#pragma unroll
      for (int k = 0; k < kEach; k += 4)
        if (place(k) < nv) *reinterpret_cast<float4 *>(y + place(k)) = *reinterpret_cast<const float4 *>(x + k);
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (place(k) < nv) y[place(k)] = x[k];
    }
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
  const int64_t want = std::max<int64_t>(1, 5ll * dev.sm_count / chunks);  // CTAs of a chunk
  const int groups = static_cast<int>(std::min<int64_t>(ntok, std::max<int64_t>(1, want / n_seq)));
  p.rows_per_cta = (ntok + groups - 1) / groups;
  p.row_groups = (ntok + p.rows_per_cta - 1) / p.rows_per_cta;
  const bool four = p.vocab % 4 == 0 && p.ld % 4 == 0 && p.out_ld % 4 == 0 && aligned16(logits) && aligned16(out);
  const cudaError_t e = launch_pdl(four ? adjust_kernel<true> : adjust_kernel<false>, dim3(n_seq * p.row_groups, chunks),
                                   dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
