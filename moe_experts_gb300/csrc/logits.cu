// Biases, penalties for repeated tokens and grammar masks on the logits of
// drafted tokens (epq_logits_adjust).
//
//   l += b(v);  seen: l = l > 0 ? l / r : l r;  n > 0: l -= f n + p;  not allowed: -inf
//
// n(v) counts the row's generated tokens v: the history behind the prompt, and
// the drafted tokens on the row's path.  A CTA takes kChunk tokens of the
// vocabulary for some rows of one sequence.  It goes through the history and
// the biases once, keeps a note for each of its tokens in shared memory, and
// lists the tokens with a note and the drafted ones.  A row is then two things
// side by side: the tokens that are not listed, of which a thread has eight and
// only the mask asks, and the list, a token a thread, with the penalties' division
// and what the path adds.  (Where each thread makes up the notes of its own
// tokens, a few of them keep all lanes of most warps dividing.)  A CTA whose
// notes are more than its threads does that all the same, and lists the drafted
// tokens alone: its lanes all have notes.  Integer counts and a maximum of
// indices do not depend on the order in which threads come, and listed tokens
// not on one another, so the result does not either.
//
// 4 x 64 rows of 128256 with a grammar and 8193 tokens of history: 60 us, 267 MB
// (4.5 TB/s, 0.66 of the copy rate): latencies, of a CTA's beginning and of a row
// (one is on its way while one is worked on), and the CTAs whose tokens are in
// the history for the most part, whose rows take 1.7 times as long.  21 rows of
// 50001: 9.7 us; one row of 128256: 4.3 us, the chain of history, notes, list, row.
// Where each thread made up its own tokens' notes 87 us; with the history asked
// for after its length 70 us.
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

// A token's note: its count, whether the prompt has it, whether it has a bias,
// whether it is drafted.
constexpr uint32_t kRead = 0x80000000u, kBiased = 0x40000000u, kDrafted = 0x20000000u, kCount = 0x1fffffffu;

struct Penalties {
  float repetition, frequency, presence;
  float inverse;  // of the repetition; 0 where it is out of the range in which quotients are corrected
};

// l / r, rounded once.  The quotient by the rounded reciprocal is off by at most
// 1.5 units; one correction by its remainder brings it within one, and from there
// the second one rounds as the division does (Markstein).  A CTA whose tokens
// mostly have a note divides eight times a thread and row.
__device__ __forceinline__ float over(float l, const Penalties &p) {
  float q = __fmul_rn(l, p.inverse);
  if (!(q > 0x1p-60f && q < 0x1p60f)) return __fdiv_rn(l, p.repetition);
  q = fmaf(fmaf(-p.repetition, q, l), p.inverse, q);
  return fmaf(fmaf(-p.repetition, q, l), p.inverse, q);
}

__device__ __forceinline__ float adjusted(float l, uint32_t w, float bias, const Penalties &p) {
  if (w & kBiased) l = __fadd_rn(l, bias);
  if (w & (kRead | kCount)) l = l > 0.0f ? over(l, p) : __fmul_rn(l, p.repetition);
  if (w & kCount)
    l = __fsub_rn(l, __fadd_rn(__fmul_rn(p.frequency, static_cast<float>(w & kCount)), p.presence));
  return l;
}

// kFour: a thread has four tokens next to one another, in 16-byte words (rows
// that begin at 16 bytes); else every 256th.
template <bool kFour>
__global__ void __launch_bounds__(kThreads, 4) adjust_kernel(const __grid_constant__ LogitsParams p) {
  constexpr int kEach = kChunk / kThreads, kRun = kFour ? 4 : 1;
  __shared__ __align__(16) uint32_t note[kChunk];
  __shared__ __align__(16) float added[kChunk];  // first 1 + the last bias entry (0: none), then that bias
  __shared__ unsigned short list[kThreads];      // places in the chunk, the drafted tokens' first
  __shared__ int drafted[kMaxTokens], many[2];   // places of the drafted tokens, or -1; listed of them, and others
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  const int s = blockIdx.x / p.row_groups, r0 = (blockIdx.x - s * p.row_groups) * p.rows_per_cta;
  const int v0 = blockIdx.y * kChunk, nv = min(kChunk, p.vocab - v0);
  const int r1 = min(r0 + p.rows_per_cta, p.ntok);
  const auto place = [&](int k) { return kFour ? 4 * (tid + kThreads * (k / 4)) + k % 4 : tid + kThreads * k; };
  const float *from = p.x + (static_cast<int64_t>(s) * p.ntok + r0) * p.ld + v0;
  float *to = p.y + (static_cast<int64_t>(s) * p.ntok + r0) * p.out_ld + v0;
  const uint32_t *allowed = p.allowed ? p.allowed + (static_cast<int64_t>(s) * p.ntok + r0) * p.words + v0 / 32 : nullptr;
  const uint64_t *mask = p.mask ? p.mask + static_cast<int64_t>(s) * p.ntok + r0 : nullptr;
  // What a thread reads of a row: its tokens' logits and words of the mask; the
  // same of its first listed token, and the path.  The next row is read while
  // one is worked on.
  struct Row {
    __align__(16) float x[kEach];
    uint32_t in[kEach / kRun];
    float l;
    uint32_t l_in;
    uint64_t path;
  } now, ahead;
  int at0 = -1;  // the thread's first listed token
  const auto load = [&](Row &row, const float *from, const uint32_t *allowed) {
#pragma unroll
    for (int k = 0; k < kEach; k += kRun) {
      row.in[k / kRun] = ~0u;
      if (place(k) >= nv) continue;
      if constexpr (kFour) *reinterpret_cast<float4 *>(row.x + k) = *reinterpret_cast<const float4 *>(from + place(k));
      else row.x[k] = from[place(k)];
      if (allowed) row.in[k / kRun] = allowed[place(k) >> 5];
    }
  };
  const auto load_listed = [&](Row &row, const float *from, const uint32_t *allowed, const uint64_t *mask, int r) {
    row.l = 0.0f, row.l_in = ~0u, row.path = ~0ull >> (63 - (r & 63));
    if (at0 < 0) return;
    row.l = from[at0];
    if (allowed) row.l_in = allowed[at0 >> 5];
    if (mask) row.path = *mask;
  };
  load(now, from, allowed);
  // all that the CTA has to know is asked for at once; a first look at the history
  // does not wait for its length
  constexpr int kLook = 16;
  const int32_t *h = p.history + static_cast<int64_t>(s) * p.max_history;
  unsigned look[kLook];
#pragma unroll
  for (int k = 0; k < kLook; ++k) look[k] = p.history && tid + k * kThreads < p.max_history ? static_cast<unsigned>(h[tid + k * kThreads]) : ~0u;
  const int32_t *ids = p.bias_ids + static_cast<int64_t>(s) * p.n_bias;
  const unsigned id0 = tid < p.n_bias ? static_cast<unsigned>(ids[tid]) : ~0u;
  const unsigned token = p.tokens && tid < p.ntok ? static_cast<unsigned>(p.tokens[static_cast<int64_t>(s) * p.ntok + tid]) : ~0u;
  const int length = p.history_len ? min(max(p.history_len[s], 0), p.max_history) : p.max_history;
  const int given = p.prompt_len ? min(max(p.prompt_len[s], 0), length) : 0;
  const int live = p.n_tok ? min(max(p.n_tok[s], 0), p.ntok) : p.ntok;
  Penalties pen = {1.0f, 0.0f, 0.0f, 1.0f};
  if (p.penalties) {
    pen = {p.penalties[3 * s], p.penalties[3 * s + 1], p.penalties[3 * s + 2], 0.0f};
    if (pen.repetition > 0x1p-30f && pen.repetition < 0x1p30f) pen.inverse = __frcp_rn(pen.repetition);
  }
  unsigned noted = 0, listed = 0;  // of the thread's tokens, those with a note, and those that the list has
  uint64_t mine = 0;  // the drafted tokens that are the thread's first listed one
  uint32_t w0 = 0;    // its note and its bias
  float b0 = 0.0f;
  if (r0 < live) {
    int *entry = reinterpret_cast<int *>(added);
    for (int i = 4 * tid; i < kChunk; i += 4 * kThreads) {
      *reinterpret_cast<uint4 *>(note + i) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4 *>(entry + i) = make_uint4(0, 0, 0, 0);
    }
    if (tid < 2) many[tid] = 0;
    if (tid < kMaxTokens) {
      const unsigned at = tid < live ? token - v0 : ~0u;
      drafted[tid] = at < static_cast<unsigned>(nv) ? static_cast<int>(at) : -1;
    }
    __syncthreads();
    if (p.history) {
      for (int i0 = tid; i0 < length; i0 += kLook * kThreads) {
        if (i0 != tid) {
#pragma unroll
          for (int k = 0; k < kLook; ++k) look[k] = i0 + k * kThreads < length ? static_cast<unsigned>(h[i0 + k * kThreads]) : ~0u;
        }
#pragma unroll
        for (int k = 0; k < kLook; ++k) {
          const unsigned at = look[k] - v0;
          if (i0 + k * kThreads >= length || at >= static_cast<unsigned>(nv)) continue;
          if (i0 + k * kThreads < given) atomicOr(&note[at], kRead);
          else atomicAdd(&note[at], 1u);
        }
      }
    }
    for (int i = tid; i < p.n_bias; i += kThreads) {
      const unsigned at = (i == tid ? id0 : static_cast<unsigned>(ids[i])) - v0;
      if (at >= static_cast<unsigned>(nv)) continue;
      atomicOr(&note[at], kBiased);
      atomicMax(&entry[at], i + 1);
    }
    if (p.tokens && tid < kMaxTokens && drafted[tid] >= 0) {
      bool first = true;
      for (int j = 0; j < tid; ++j) first = first && drafted[j] != drafted[tid];
      if (first) {
        atomicOr(&note[drafted[tid]], kDrafted);
        list[atomicAdd(&many[0], 1)] = static_cast<unsigned short>(drafted[tid]);
      }
    }
    __syncthreads();
    const int first = many[0];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const uint32_t w = note[place(k)];
      if (w & ~kDrafted) noted |= 1u << k;
      if (w & kDrafted) listed |= 1u << k;
      if (w & kBiased) added[place(k)] = p.bias[static_cast<int64_t>(s) * p.n_bias + entry[place(k)] - 1];
    }
    noted &= ~listed;
    if (noted) atomicAdd(&many[1], __popc(noted));
    __syncthreads();
    const bool fits = first + many[1] <= kThreads;
    int end = first;
    if (fits) {
      end = first + many[1];
      __syncthreads();  // every thread has read what is counted down here
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (noted >> k & 1) list[first - 1 + atomicSub(&many[1], 1)] = static_cast<unsigned short>(place(k));
      listed |= noted, noted = 0;
      __syncthreads();
    }
    if (tid < end) at0 = list[tid], w0 = note[at0], b0 = added[at0];
    if (tid < first)
      for (int j = 0; j < kMaxTokens; ++j) mine |= static_cast<uint64_t>(drafted[j] == at0) << j;
    load_listed(now, from, allowed, mask, r0);
  }
  const auto work = [&](int r, Row &now, Row &ahead) {
    if (r + 1 < r1) {
      const uint32_t *next = allowed ? allowed + p.words : nullptr;
      load(ahead, from + p.ld, next);
      load_listed(ahead, from + p.ld, next, mask ? mask + 1 : nullptr, r + 1);
    }
    if (r < live) {
      if (at0 >= 0) {
        const float l = adjusted(now.l, w0 + __popcll(now.path & mine), b0, pen);
        to[at0] = now.l_in >> (at0 & 31) & 1 ? l : -INFINITY;
      }
      if (noted) {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          if (noted >> k & 1) now.x[k] = adjusted(now.x[k], note[place(k)], added[place(k)], pen);
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (!(now.in[k / kRun] >> (place(k) & 31) & 1)) now.x[k] = -INFINITY;
    }
    if (r < live || p.x != p.y) {
#pragma unroll
      for (int k = 0; k < kEach; k += kRun) {
        const int at = place(k);
        if (at >= nv) continue;
        if (kFour && (r >= live || !(listed >> k & 15))) {
          *reinterpret_cast<float4 *>(to + at) = *reinterpret_cast<const float4 *>(now.x + k);
        } else {
#pragma unroll
          for (int i = 0; i < kRun; ++i)
            if (r >= live || !(listed >> (k + i) & 1)) to[at + i] = now.x[k + i];
        }
      }
    }
    from += p.ld, to += p.out_ld;
    if (allowed) allowed += p.words;
    if (mask) ++mask;
  };
  for (int r = r0; r < r1; r += 2) {  // (no copy: the row ahead has the time of a whole row to come)
    work(r, now, ahead);
    if (r + 1 < r1) work(r + 1, ahead, now);
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
  // rows share the pass over the history, but all SMs have CTAs: 8 for each of
  // four that fit at a time even out the CTAs with long lists (4 x 64 rows: 4 for
  // each SM 91 us, 8 60, 16 65)
  const int64_t want = std::max<int64_t>(1, 8ll * dev.sm_count / chunks);  // CTAs of a chunk
  const int groups = static_cast<int>(std::min<int64_t>(ntok, std::max<int64_t>(1, want / n_seq)));
  p.rows_per_cta = (ntok + groups - 1) / groups;
  p.row_groups = (ntok + p.rows_per_cta - 1) / p.rows_per_cta;
  const bool four = p.vocab % 4 == 0 && p.ld % 4 == 0 && p.out_ld % 4 == 0 && aligned16(logits) && aligned16(out);
  const cudaError_t e = launch_pdl(four ? adjust_kernel<true> : adjust_kernel<false>, dim3(n_seq * p.row_groups, chunks),
                                   dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
