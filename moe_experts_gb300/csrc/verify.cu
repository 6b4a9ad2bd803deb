// Acceptance of drafted tokens against the target's probabilities
// (epq_verify_tree).
//
// Two launches: row_stats_kernel reads every logits row once (maximum with
// its lowest index, sum of exponentials), walk_kernel goes down the tree of
// one sequence, one CTA per sequence.
//
// The weights w(v) = exp((l_v - max) / T) of a row in which the walk rejects
// or ends are formed in double precision and summed as 64-bit integers in
// units of 2^-44: the sums do not depend on their order, and the drawn token
// (a comparison of a partial sum with u times the total) is settled to about
// 2^-45 of the largest weight.  vocab <= 2^18 keeps every sum below 2^62.
#include <cmath>

#include "pages.cuh"

namespace epq {
namespace {

constexpr int kStatThreads = 256;
constexpr int kWalkThreads = 1024;
constexpr int64_t kMaxVocab = 262144;
constexpr double kUnit = 17592186044416.0;  // 2^44

struct VerifyParams {
  const float *logits, *draft, *u;
  const int32_t *tokens, *parent, *n_tok;
  int64_t ld, draft_ld;
  int vocab, n_seq, ntok, greedy;
  float temperature;
  int32_t *path, *n_accept, *next_token;
  float *lse;
  float *row_max;  // workspace: [n_seq * ntok]
  float *row_sum;
  int32_t *row_arg;
};

__device__ __forceinline__ int tree_size(const int32_t *n_tok, int s, int ntok) {
  return n_tok ? min(max(n_tok[s], 0), ntok) : ntok;
}

// Larger value first, then lower index.
__device__ __forceinline__ void take_max(float &m, int &at, float m2, int at2) {
  if (m2 > m || (m2 == m && at2 < at)) m = m2, at = at2;
}

__global__ void __launch_bounds__(kStatThreads) row_stats_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ float sm[8];
  __shared__ int si[8];
  __shared__ float ss[8];
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x / p.ntok, i = blockIdx.x % p.ntok;
  if (i >= tree_size(p.n_tok, s, p.ntok)) {
    if (threadIdx.x == 0 && p.lse) p.lse[blockIdx.x] = 0.0f;
    return;
  }
  const float *row = p.logits + blockIdx.x * p.ld;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY;
  int at = 0;
  for (int v = threadIdx.x; v < p.vocab; v += kStatThreads) take_max(m, at, row[v], v);
  for (int o = 16; o > 0; o >>= 1)
    take_max(m, at, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, at, o));
  if (lane == 0) sm[warp] = m, si[warp] = at;
  __syncthreads();
  m = sm[0], at = si[0];
  for (int w = 1; w < 8; ++w) take_max(m, at, sm[w], si[w]);
  const float inv_t = p.greedy ? 1.0f : 1.0f / p.temperature;
  float z = 0.0f;
  for (int v = threadIdx.x; v < p.vocab; v += kStatThreads) z += expf((row[v] - m) * inv_t);
  z = warp_sum_xor<32>(z);
  if (lane == 0) ss[warp] = z;
  __syncthreads();
  if (threadIdx.x == 0) {
    z = 0.0f;
    for (int w = 0; w < 8; ++w) z += ss[w];
    p.row_max[blockIdx.x] = m;
    p.row_sum[blockIdx.x] = z;
    p.row_arg[blockIdx.x] = at;
    if (p.lse) p.lse[blockIdx.x] = m * inv_t + logf(z);
  }
}

__device__ __forceinline__ long long block_sum(long long x, long long *sums) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
  for (int w = 0; w < kWalkThreads / 32; ++w) x += sums[w];
  return x;
}

__global__ void __launch_bounds__(kWalkThreads) walk_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ long long sums[kWalkThreads / 32];
  __shared__ int gone[kMaxTree];  // rejected tokens of the current node (no draft)
  __shared__ int drawn;
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x, tid = threadIdx.x;
  const int n = tree_size(p.n_tok, s, p.ntok);
  const int base = s * p.ntok;
  int32_t *path = p.path + base;
  for (int i = tid; i < p.ntok; i += kWalkThreads)
    if (i >= 1 || n == 0) path[i] = -1;
  if (n == 0) {
    if (tid == 0) p.n_accept[s] = 0, p.next_token[s] = -1;
    return;
  }
  const bool use_draft = p.draft != nullptr && !p.greedy;
  const double inv_t = p.greedy ? 1.0 : 1.0 / static_cast<double>(p.temperature);
  int cur = 0, count = 1, n_gone = 0;
  const float *row = p.logits + static_cast<int64_t>(base) * p.ld;
  const float *q = use_draft ? p.draft + static_cast<int64_t>(base) * p.draft_ld : nullptr;
  float m = p.row_max[base];
  double R = p.row_sum[base];  // in units of the largest weight
  double S = 0.0;
  auto weight = [&](int v) { return exp((static_cast<double>(row[v]) - static_cast<double>(m)) * inv_t); };
  auto left = [&](int v) {  // r(v) in units of 2^-44
    double w = weight(v);
    if (use_draft) w = fmax(w - S * static_cast<double>(q[v]), 0.0);
    for (int k = 0; k < n_gone; ++k)
      if (gone[k] == v) w = 0.0;
    return __double2ll_rn(w * kUnit);
  };
  auto total = [&]() {
    long long t = 0;
    for (int v = tid; v < p.vocab; v += kWalkThreads) t += left(v);
    return block_sum(t, sums);
  };
  if (tid == 0) path[0] = 0;
  __syncthreads();
  for (int i = 1; i < n; ++i) {  // every thread takes the same decisions
    if (p.parent[base + i] != cur) continue;
    const int x = p.tokens[base + i];
    const bool known = x >= 0 && x < p.vocab;
    bool yes = false;
    if (p.greedy) {
      yes = x == p.row_arg[base + cur];
    } else if (known) {
      const double here = static_cast<double>(left(x)) / kUnit;
      const double qx = use_draft ? static_cast<double>(q[x]) : 1.0;
      yes = static_cast<double>(p.u[base + i]) * qx * R < here;
    }
    if (yes) {
      __syncthreads();  // `gone` is no longer read
      cur = i;
      n_gone = 0;
      S = 0.0;
      row = p.logits + static_cast<int64_t>(base + i) * p.ld;
      if (use_draft) q = p.draft + static_cast<int64_t>(base + i) * p.draft_ld;
      m = p.row_max[base + i];
      R = p.row_sum[base + i];
      if (tid == 0) path[count] = i;
      ++count;
    } else if (!p.greedy && use_draft) {
      if (S == 0.0) R = static_cast<double>(total()) / kUnit;  // the exact sum of the row's weights
      const double kept = S;
      S += R;
      const double less = static_cast<double>(total()) / kUnit;
      if (less > 0.0) R = less;
      else S = kept;
    } else if (!p.greedy && known) {
      R -= static_cast<double>(left(x)) / kUnit;
      __syncthreads();
      if (tid == 0) gone[n_gone] = x;
      ++n_gone;
      __syncthreads();
    }
  }
  // the next token
  int next = p.row_arg[base + cur];
  if (!p.greedy) {
    const int per = (p.vocab + kWalkThreads - 1) / kWalkThreads;  // consecutive entries of a thread
    const int v0 = min(tid * per, p.vocab), v1 = min(v0 + per, p.vocab);
    long long mine = 0;
    for (int v = v0; v < v1; ++v) mine += left(v);
    const long long all = block_sum(mine, sums);
    // exclusive prefix of the thread's entries
    long long before = mine;
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    before -= mine;
    for (int w = 0; w < warp; ++w) before += sums[w];
    if (tid == 0) drawn = next;
    __syncthreads();
    const double t = static_cast<double>(p.u[base]) * static_cast<double>(all);
    if (static_cast<double>(before) <= t && static_cast<double>(before + mine) > t) {
      for (int v = v0; v < v1; ++v) {
        before += left(v);
        if (static_cast<double>(before) > t) {
          drawn = v;
          break;
        }
      }
    }
    __syncthreads();
    next = drawn;
  }
  if (tid == 0) p.n_accept[s] = count, p.next_token[s] = next;
}

__global__ void __launch_bounds__(64) tree_mask_kernel(const int32_t *__restrict__ parent, int n_seq, int ntok,
                                                       uint64_t *__restrict__ mask) {
  __shared__ int up[kMaxTree];
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x, i = threadIdx.x;
  if (i < ntok) up[i] = parent[s * ntok + i];
  __syncthreads();
  if (i >= ntok) return;
  uint64_t m = 0;
  for (int c = i; c >= 0;) {  // indices fall, so this ends
    m |= 1ull << c;
    c = up[c] < c ? up[c] : -1;
  }
  mask[s * ntok + i] = m;
}

bool device_ok() {
  DeviceInfo dev;
  return current_device(&dev) && dev.major * 10 + dev.minor >= 100;
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" epq_status epq_tree_mask(const int32_t *parent, int n_seq, int ntok, uint64_t *mask, epq_stream_t stream) {
  if (!parent || !mask) return EPQ_ERR_ARG;
  if (n_seq < 1 || n_seq > kMaxSeq || ntok < 1 || ntok > kMaxTree) return EPQ_ERR_SHAPE;
  if (!device_ok()) return EPQ_ERR_DEVICE;
  const cudaError_t e = launch_pdl(tree_mask_kernel, dim3(n_seq), dim3(64), 0, reinterpret_cast<cudaStream_t>(stream),
                                   parent, n_seq, ntok, mask);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}

extern "C" size_t epq_verify_tree_workspace_bytes(int n_seq, int ntok, int64_t vocab) {
  if (n_seq < 1 || n_seq > kMaxSeq || ntok < 1 || ntok > kMaxTree || vocab < 1 || vocab > kMaxVocab) return 0;
  return 3 * sizeof(float) * static_cast<size_t>(n_seq) * ntok;
}

extern "C" epq_status epq_verify_tree(const float *logits, int64_t vocab, const int32_t *tokens, const int32_t *parent,
                                      const float *u, int n_seq, int ntok, const epq_verify_opts *opts, int32_t *path,
                                      int32_t *n_accept, int32_t *next_token, float *lse, void *ws, size_t ws_bytes,
                                      epq_stream_t stream) {
  if (!logits || !tokens || !parent || !path || !n_accept || !next_token) return EPQ_ERR_ARG;
  const size_t need = epq_verify_tree_workspace_bytes(n_seq, ntok, vocab);
  if (!need) return EPQ_ERR_SHAPE;
  VerifyParams p = {};
  p.temperature = opts ? opts->temperature : 1.0f;
  if (!(p.temperature >= 0.0f) || std::isinf(p.temperature)) return EPQ_ERR_ARG;
  p.greedy = p.temperature == 0.0f;
  if (!p.greedy && !u) return EPQ_ERR_ARG;
  p.ld = opts && opts->ld ? opts->ld : vocab;
  p.draft_ld = opts && opts->draft_ld ? opts->draft_ld : vocab;
  if (p.ld < vocab || p.draft_ld < vocab) return EPQ_ERR_SHAPE;
  if (!ws || ws_bytes < need) return EPQ_ERR_WORKSPACE;
  if (!aligned16(logits) || !aligned16(ws) || (opts && opts->draft && !aligned16(opts->draft))) return EPQ_ERR_ALIGN;
  if (!device_ok()) return EPQ_ERR_DEVICE;
  p.logits = logits;
  p.draft = opts ? opts->draft : nullptr;
  p.u = u;
  p.tokens = tokens;
  p.parent = parent;
  p.n_tok = opts ? opts->n_tok : nullptr;
  p.vocab = static_cast<int>(vocab);
  p.n_seq = n_seq;
  p.ntok = ntok;
  p.path = path;
  p.n_accept = n_accept;
  p.next_token = next_token;
  p.lse = lse;
  p.row_max = static_cast<float *>(ws);
  p.row_sum = p.row_max + static_cast<size_t>(n_seq) * ntok;
  p.row_arg = reinterpret_cast<int32_t *>(p.row_sum + static_cast<size_t>(n_seq) * ntok);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(row_stats_kernel, dim3(n_seq * ntok), dim3(kStatThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(walk_kernel, dim3(n_seq), dim3(kWalkThreads), 0, s, p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
