// Acceptance of drafted tokens against the target's probabilities
// (epq_verify_tree).
//
// Two launches.  row_stats_kernel reads every logits row once, in chunks of
// CTAs: maximum with its lowest index and the sum of exponentials (float32,
// relative to the chunk's maximum).  walk_kernel joins them and goes down the
// tree, one thread-block cluster per sequence; warp 0 of every CTA takes the
// same decisions from the same numbers.  An acceptance needs only w(x) of the
// drafted token, which the CTA gathers for all tokens at the start; the row
// itself is read again only where a draft row has to be subtracted after a
// rejection, where a given child is judged after another was taken out, where
// u is within 2^-16 of a child's border, and once to draw the next token (its
// weights then stay in shared memory).
//
// Measured (128256 tokens, both launches from a graph): one row 12.5 us, of
// which the walk's dependent steps are the larger part (with 8 CTAs per
// sequence that read the row again to draw: 25 us); 8 rows with draft
// probabilities 21 us; 4 sequences of 64 rows 52 us, 131 MB (51 to 55 with the
// rejections that the inputs make).
//
// Drawing compares a partial sum of up to 2^18 weights with u times their
// total.  The weights w(v) = exp((l_v - max) / T) are therefore formed to
// 2^-29 of themselves (root mean square 2^-31.5) and summed as 64-bit integers
// in units of 2^-44 (0 below half a unit): the sums do not depend on their
// order, and a wrong neighbour needs u within 4e-9 of a boundary.  With t =
// (l - max) log2(e) / T = n + j / 32 + g (n, j integers, |g| <= 1/64,
// everything that float32 loses of l - max and of the product kept in a second
// float)
//   w = 2^n 2^(j/32) (1 + (z + z^2/2 + z^3/6 + ...)),  z = g ln 2,
// a table entry of 62 bits plus a small float, shifted right by 18 - n.  (GB300
// has two double-precision lanes per SM and clock; the same pass in double
// precision took 0.8 ms for 128256 tokens.)
#include <algorithm>
#include <cmath>

#include "pages.cuh"

namespace epq {
namespace {

constexpr int kStatThreads = 256;
constexpr int kWalkThreads = 512;
constexpr int kWalkWarps = kWalkThreads / 32;
constexpr int kWalkCluster = 16;  // CTAs of one sequence; more than 8 need the kernel's opt-in
constexpr int kGroup = 256;       // entries that a warp reads at a time
constexpr int64_t kMaxVocab = 262144;
constexpr double kUnit = 17592186044416.0;  // 2^44
// A row's float32 sum of exponentials is within 2^-16 of the integer weights'
// sum: up to 93 roundings of 2^-24 on the way of a term (23 in its chunk, 10
// joins of 7), 2^-22 of ex2.approx, and arguments of up to 64 binary orders that
// are off by 3 x 2^-24 of themselves, all together below 1.4e-5.
constexpr float kSumError = 1.52587890625e-5f;
// CTAs from which row_stats_kernel takes long chunks (two per SM of a GB300)
constexpr int64_t kManyChunks = 304;

struct VerifyParams {
  const float *logits, *draft, *u;
  const int32_t *tokens, *parent, *n_tok;
  int64_t ld, draft_ld;
  int vocab, n_seq, ntok, greedy, splits;
  float c_hi, c_lo;  // log2(e) / temperature in two parts
  float inv_t;
  int32_t *path, *n_accept, *next_token;
  float *lse;
  float *part_max;  // workspace: [rows][splits]
  float *part_sum;
  int32_t *part_arg;
  unsigned long long table[32];  // 2^(j/32) in units of 2^-62
};

__device__ __forceinline__ int tree_size(const int32_t *n_tok, int s, int ntok) {
  return n_tok ? min(max(n_tok[s], 0), ntok) : ntok;
}

// Larger value first, then lower index.
__device__ __forceinline__ void take_max(float &m, int &at, float m2, int at2) {
  if (m2 > m || (m2 == m && at2 < at)) m = m2, at = at2;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Sum over maxima: z relative to m joined with z2 relative to m2.
__device__ __forceinline__ float join_sum(float m, float z, float top, float c) {
  return m == -INFINITY ? 0.0f : z * exp2_fast((m - top) * c);
}

// Grid (splits, rows).  A CTA reads 1024 VEC consecutive floats of a row,
// 16 bytes at a time from 16-byte boundaries (a row may begin between two).
// Bound by what a CTA does after its loads have landed, over four CTAs an SM:
// 131 MB in 26.5 us, 5.0 TB/s (0.73 of the copy bandwidth); chunks of 4096 the
// same, of 16384 41 us.
template <int VEC>
__global__ void __launch_bounds__(kStatThreads) row_stats_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ float sm[8], ss[8];
  __shared__ int si[8];
  pdl_launch_dependents();
  pdl_wait();
  const int r = blockIdx.y;
  if (r % p.ntok >= tree_size(p.n_tok, r / p.ntok, p.ntok)) return;
  const float *row = p.logits + static_cast<int64_t>(r) * p.ld;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(row) / 4 & 3);  // floats past a boundary
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float4 x[VEC];
  const int v0 = blockIdx.x * (1024 * VEC) - shift + 4 * static_cast<int>(threadIdx.x);
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const int v = v0 + 1024 * k;
    if (v >= 0 && v + 3 < p.vocab) {
      x[k] = __ldg(reinterpret_cast<const float4 *>(row + v));
    } else {
      x[k].x = v >= 0 && v < p.vocab ? row[v] : -INFINITY;
      x[k].y = v + 1 >= 0 && v + 1 < p.vocab ? row[v + 1] : -INFINITY;
      x[k].z = v + 2 >= 0 && v + 2 < p.vocab ? row[v + 2] : -INFINITY;
      x[k].w = v + 3 >= 0 && v + 3 < p.vocab ? row[v + 3] : -INFINITY;
    }
  }
  float mine = -INFINITY;
#pragma unroll
  for (int k = 0; k < VEC; ++k) mine = fmaxf(mine, fmaxf(fmaxf(x[k].x, x[k].y), fmaxf(x[k].z, x[k].w)));
  float m = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sm[warp] = m;
  __syncthreads();
  m = sm[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) m = fmaxf(m, sm[w]);
  const float ref = m == -INFINITY ? 0.0f : m;
  float z = 0.0f;
#pragma unroll
  for (int k = 0; k < VEC; ++k)
    z += (exp2_fast((x[k].x - ref) * p.c_hi) + exp2_fast((x[k].y - ref) * p.c_hi)) +
         (exp2_fast((x[k].z - ref) * p.c_hi) + exp2_fast((x[k].w - ref) * p.c_hi));
  z = warp_sum_xor<32>(z);
  // the lowest index of the maximum, where a thread of the warp has it
  int at = 0x7fffffff;
  if (__any_sync(0xffffffffu, mine == m)) {
#pragma unroll
    for (int k = VEC - 1; k >= 0; --k) {
      const int v = v0 + 1024 * k;
      if (x[k].w == m) at = v + 3;
      if (x[k].z == m) at = v + 2;
      if (x[k].y == m) at = v + 1;
      if (x[k].x == m) at = v;
    }
    at = __reduce_min_sync(0xffffffffu, m == -INFINITY ? 0x7fffffff : at);
  }
  if (lane == 0) ss[warp] = z, si[warp] = at;
  __syncthreads();
  if (threadIdx.x == 0) {
    z = 0.0f;
    for (int w = 0; w < 8; ++w) {
      z += ss[w];
      at = min(at, si[w]);
    }
    const int64_t i = static_cast<int64_t>(r) * p.splits + blockIdx.x;
    p.part_max[i] = m;
    p.part_sum[i] = z;
    p.part_arg[i] = at;
  }
}

struct Table {
  unsigned long long t[32];
  float f[32];  // 2^(j/32) in units of 2^-36
};

// exp((l - m) / T) in units of 2^-44, l <= m (see the head of the file).
__device__ __forceinline__ long long weight_fixed(float l, float m, float c_hi, float c_lo, const Table &tab) {
  const float d = l - m;
  float t = d * c_hi;
  if (!(t >= -45.015625f)) return 0;  // below half a unit (the shift is 63 at most), or a NaN
  const float b = d - l;
  const float e = (l - (d - b)) + (-m - b);  // l - m = d + e
  const float te = fmaf(d, c_hi, -t) + fmaf(d, c_lo, e * c_hi);
  const float k = rintf(t * 32.0f);
  const float g = fmaf(k, -0.03125f, t);
  const float z = fmaf(g, 0.693147182464599609375f, fmaf(te, 0.693147182464599609375f, g * -1.904654323148236e-09f));
  const float x = fmaf(z * z, fmaf(z, fmaf(z, 0.041666667f, 0.16666667f), 0.5f), z);
  const int ki = static_cast<int>(k), j = ki & 31;
  const long long f = static_cast<long long>(tab.t[j]) + (static_cast<long long>(__float2int_rn(x * tab.f[j])) << 26);
  const int s = 18 - (ki >> 5);
  return static_cast<long long>((static_cast<unsigned long long>(f) + (1ull << (s - 1))) >> s);
}

// max(w - S q, 0) in the same units, S = s_hi + s_lo.
__device__ __forceinline__ long long subtract_fixed(long long w, float s_hi, float s_lo, float q) {
  const float a = s_hi * q;
  if (!(a < 2.0f)) return 0;  // w <= 1
  const float ae = fmaf(s_hi, q, -a) + s_lo * q;
  const int i = __float2int_rn(a * 268435456.0f);  // 2^28
  const float rest = fmaf(static_cast<float>(i >> 8), -9.5367431640625e-7f, a) -
                     static_cast<float>(i & 255) * 3.7252902984619140625e-9f + ae;
  const long long v = w - (static_cast<long long>(i) << 16) - __float2int_rn(rest * 17592186044416.0f);
  return v > 0 ? v : 0;
}

// Consecutive entries of a row that one warp of a cluster holds.
__host__ __device__ inline int walk_entries(int vocab) {
  const int warps = kWalkCluster * kWalkWarps;
  return ((vocab + warps - 1) / warps + kGroup - 1) / kGroup * kGroup;
}

// One cluster per sequence.
__global__ void __launch_bounds__(kWalkThreads) walk_kernel(const __grid_constant__ VerifyParams p) {
  extern __shared__ __align__(16) uint8_t smem[];  // weights, draft row
  __shared__ Table tab;
  __shared__ float top[kMaxTree], sum[kMaxTree], lx[kMaxTree], qx[kMaxTree], us[kMaxTree];
  __shared__ int arg[kMaxTree], tok[kMaxTree], up[kMaxTree], gone[kMaxTree];
  __shared__ long long warp_sum[kWalkWarps];
  __shared__ long long cta_sum[2][kWalkCluster];
  __shared__ struct {
    int state, cur, n_gone, filled, next, draw;
    float s_hi, s_lo;
    long long u_all;
  } ask;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int s = blockIdx.x / kWalkCluster;
  if (tid < 32) {
    tab.t[tid] = p.table[tid];
    tab.f[tid] = static_cast<float>(static_cast<double>(p.table[tid]) * 1.4901161193847656e-08);  // 2^-26
  }
  pdl_launch_dependents();
  pdl_wait();
  const int n = tree_size(p.n_tok, s, p.ntok);
  const int base = s * p.ntok;
  int32_t *path = p.path + base;
  const bool writer = rank == 0;
  if (writer) {
    for (int i = tid; i < p.ntok; i += kWalkThreads) {
      if (i >= n && p.lse) p.lse[base + i] = 0.0f;
      if (i >= 1 || n == 0) path[i] = -1;
    }
    if (n == 0 && tid == 0) p.n_accept[s] = 0, p.next_token[s] = -1;
  }
  if (n == 0) return;  // the whole cluster
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const bool use_draft = p.draft != nullptr && !p.greedy;
  // the drafted tokens' logits and draft probabilities in their parents' rows
  if (tid < n) {
    const int x = p.tokens[base + tid], a = p.parent[base + tid];
    tok[tid] = x;
    up[tid] = a;
    us[tid] = p.greedy ? 0.0f : fminf(fmaxf(p.u[base + tid], 0.0f), 0.999999940395355225f);  // [0, 1); NaN: 0
    const bool known = tid > 0 && a >= 0 && a < tid && x >= 0 && x < p.vocab;
    lx[tid] = known ? p.logits[static_cast<int64_t>(base + a) * p.ld + x] : -INFINITY;
    qx[tid] = known && use_draft ? p.draft[static_cast<int64_t>(base + a) * p.draft_ld + x] : 1.0f;
  }
  // A row's chunks joined by half a warp (a whole one when there are more than
  // 16), so that 64 rows take two rounds of loads.
  {
    const int width = p.splits <= 16 ? 16 : 32, rows = 32 / width, l = lane & (width - 1);
    for (int r0 = warp * rows; r0 < n; r0 += kWalkWarps * rows) {  // the same turns for both halves
      const int r = r0 + lane / width;
      const int64_t i = static_cast<int64_t>(base + min(r, n - 1)) * p.splits;
      float m = -INFINITY, z = 0.0f;
      int at = 0x7fffffff;
      auto join = [&](float m2, float z2, int at2) {
        const float up = fmaxf(m, m2);
        z = join_sum(m, z, up, p.c_hi) + join_sum(m2, z2, up, p.c_hi);
        take_max(m, at, m2, at2);
      };
      for (int k = l; k < p.splits; k += width) join(p.part_max[i + k], p.part_sum[i + k], p.part_arg[i + k]);
      for (int o = width / 2; o > 0; o >>= 1)
        join(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, z, o), __shfl_xor_sync(0xffffffffu, at, o));
      if (l == 0 && r < n) {
        top[r] = m;
        sum[r] = z;
        arg[r] = at < p.vocab ? at : 0;  // a row without a finite logit
        if (writer && p.lse) p.lse[base + r] = m * p.inv_t + logf(z);
      }
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA has started: its shared memory may be written

  // A warp has `per` consecutive entries of a row (whole groups).  The weights
  // of the current row, once they are needed, and its draft row stay in shared
  // memory.
  const int per = walk_entries(p.vocab);
  const int w0 = min((static_cast<int>(rank) * kWalkWarps + warp) * per, p.vocab), w1 = min(w0 + per, p.vocab);
  long long *w_row = reinterpret_cast<long long *>(smem) + warp * per;
  float *q_row = reinterpret_cast<float *>(smem + 8 * kWalkWarps * per) + warp * per;
  int phase = 0;
  // sum of r(v) over the row, in units of 2^-44; warp_sum and cta_sum[phase]
  // keep the parts
  auto total = [&](int cur, bool filled, float s_hi, float s_lo, int n_gone) {
    const float m = top[cur];
    const float *row = p.logits + static_cast<int64_t>(base + cur) * p.ld;
    const float *q = use_draft ? p.draft + static_cast<int64_t>(base + cur) * p.draft_ld : nullptr;
    long long t = 0;
    if (filled) {
#pragma unroll 4
      for (int i = lane; i < w1 - w0; i += 32)
        t += use_draft ? subtract_fixed(w_row[i], s_hi, s_lo, q_row[i]) : w_row[i];
    } else {  // S is 0
      for (int g = lane; g < w1 - w0; g += kGroup) {
        float l[kGroup / 32], d[kGroup / 32];
#pragma unroll
        for (int j = 0; j < kGroup / 32; ++j) {
          const bool in = g + 32 * j < w1 - w0;
          l[j] = in ? __ldg(row + w0 + g + 32 * j) : -INFINITY;
          d[j] = in && use_draft ? __ldg(q + w0 + g + 32 * j) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kGroup / 32; ++j) {  // the slice holds whole groups
          const long long w = weight_fixed(l[j], m, p.c_hi, p.c_lo, tab);
          w_row[g + 32 * j] = w;
          if (use_draft) q_row[g + 32 * j] = d[j];
          t += w;
        }
      }
    }
    __syncwarp();
    for (int k = 0; k < n_gone; ++k) {
      const int i = gone[k] - w0;
      if (i < 0 || i >= w1 - w0) continue;
      if (lane == 0) t -= w_row[i], w_row[i] = 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    phase ^= 1;
    if (lane == 0) warp_sum[warp] = t;
    __syncthreads();
    if (tid < kWalkCluster) {
      t = 0;
      for (int w = 0; w < kWalkWarps; ++w) t += warp_sum[w];
      uint32_t remote;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(remote)
                   : "r"(smem_addr(&cta_sum[phase][rank])), "r"(static_cast<uint32_t>(tid)));
      asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(remote), "l"(t) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    t = 0;
    for (int c = 0; c < kWalkCluster; ++c) t += cta_sum[phase][c];
    return t;
  };
  // The walk: warp 0 takes the decisions (they are scalar, some in double
  // precision, of which an SM has two lanes) and asks all warps for a sum
  // where it needs one.  A row's sum from row_stats_kernel (kSumError) decides
  // where that error does not matter; a child nearer to its border, one that a
  // draft row has to be subtracted for and one after a given child that was
  // taken out are judged by the integer sum.
  // state 1: the sum of what is left wanted (S as it is), 2: of what a draft row leaves, 3: to draw from
  int cur = 0, count = 1, n_gone = 0, i = 1, state = 0;
  double R = 0.0, S = 0.0, kept = 0.0;  // in units of the largest weight; R once it is exact
  long long all = -1;                   // the last sum, while it is that of the current state
  long long left = 0;                   // R in units of 2^-44
  bool exact = false, filled = false, rejected = false;
  if (writer && tid == 0) path[0] = 0;
  constexpr double kInv = 1.0 / kUnit;
  for (;;) {
    if (warp == 0) {
      const bool done = state == 3;
      if (state == 1 || (state == 2 && all > 0)) {
        left = all;
        R = static_cast<double>(left) * kInv;
        exact = true;
      } else if (state == 2) {
        S = kept, all = -1;
      }
      state = 0;
      for (; i < n; ++i) {
        if (up[i] != cur) continue;
        const int x = tok[i];
        const bool known = x >= 0 && x < p.vocab;
        bool yes = false;
        long long here = 0;  // r(x) without a draft row
        if (p.greedy) {
          yes = x == arg[cur];
        } else if (known && !rejected) {
          here = weight_fixed(lx[i], top[cur], p.c_hi, p.c_lo, tab);
          for (int k = 0; k < n_gone; ++k)
            if (gone[k] == x) here = 0;
          if (!exact) {
            const float w = static_cast<float>(here) * static_cast<float>(kInv), bar = us[i] * qx[i] * sum[cur];
            yes = bar < w * (1.0f - kSumError);
            if (here > 0 && (n_gone > 0 || !(yes || bar > w * (1.0f + kSumError)))) state = 1;
          } else {
            double r = static_cast<double>(here) * kInv;
            if (use_draft) r = fmax(r - S * static_cast<double>(qx[i]), 0.0);
            yes = static_cast<double>(us[i]) * static_cast<double>(qx[i]) * R < r;
          }
        }
        if (state == 0 && !p.greedy && use_draft && !exact && !yes) state = 1, rejected = true;
        if (state == 1) break;  // and this child again
        if (yes) {
          cur = i;
          n_gone = 0;
          S = 0.0;
          all = -1;
          exact = filled = false;
          if (writer && lane == 0) path[count] = i;
          ++count;
        } else if (!p.greedy && use_draft) {
          rejected = false;
          kept = S;
          S += R;
          state = 2;
          ++i;
          break;
        } else if (!p.greedy && here > 0) {  // taken out
          if (exact) {  // R is worked out before the next child otherwise
            left -= here;
            R = static_cast<double>(left) * kInv;
          }
          all = -1;
          __syncwarp();
          if (lane == 0) gone[n_gone] = x;
          ++n_gone;
          __syncwarp();
        }
      }
      if (state == 0 && !done && !p.greedy && all < 0) state = 3;
      if (lane == 0) {
        const float s_hi = static_cast<float>(S);
        ask.state = state;
        ask.cur = cur;
        ask.n_gone = n_gone;
        ask.filled = filled;
        ask.s_hi = s_hi;
        ask.s_lo = static_cast<float>(S - static_cast<double>(s_hi));
        ask.u_all = static_cast<long long>(floor(static_cast<double>(us[0]) * static_cast<double>(all)));
        ask.next = arg[cur];
        ask.draw = !p.greedy && all > 0;
        if (state == 0 && writer) p.n_accept[s] = count;
      }
    }
    __syncthreads();
    if (ask.state == 0) break;
    all = total(ask.cur, ask.filled, ask.s_hi, ask.s_lo, ask.n_gone);
    filled = true;
  }
  if (!ask.draw) {
    if (writer && tid == 0) p.next_token[s] = ask.next;
  } else {
    // the entry where the running sum passes t: its CTA, its warp, its place
    const long long t = ask.u_all;
    long long at = 0;
    for (uint32_t c = 0; c < rank; ++c) at += cta_sum[phase][c];
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    if (at <= t && t < at + warp_sum[warp]) {
      for (int v = lane; v - lane < w1 - w0; v += 32) {
        long long x = 0;
        if (v < w1 - w0) x = ask.s_hi > 0.0f ? subtract_fixed(w_row[v], ask.s_hi, ask.s_lo, q_row[v]) : w_row[v];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at + x > t);
        if (past) {
          if (lane == __ffs(past) - 1) p.next_token[s] = w0 + v;
          break;
        }
        at += __shfl_sync(0xffffffffu, x, 31);
      }
    }
  }
  // no CTA leaves while another may still write into its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// Chunks of a row: long ones where there are rows enough to fill the GPU.
static int64_t stats_chunk(int64_t rows, int64_t vocab) {
  return rows * ((vocab + 8191) / 8192) >= kManyChunks ? 8192 : 2048;
}

static int64_t stats_splits(int64_t rows, int64_t vocab) {
  const int64_t c = stats_chunk(rows, vocab);
  return (vocab + 3 + c - 1) / c;  // up to 3 floats of a chunk lie before the row
}

extern "C" size_t epq_verify_tree_workspace_bytes(int n_seq, int ntok, int64_t vocab) {
  if (n_seq < 1 || n_seq > kMaxSeq || ntok < 1 || ntok > kMaxTree || vocab < 1 || vocab > kMaxVocab) return 0;
  const int64_t rows = static_cast<int64_t>(n_seq) * ntok;
  return 3 * sizeof(float) * static_cast<size_t>(rows * stats_splits(rows, vocab));
}

extern "C" epq_status epq_verify_tree(const float *logits, int64_t vocab, const int32_t *tokens, const int32_t *parent,
                                      const float *u, int n_seq, int ntok, const epq_verify_opts *opts, int32_t *path,
                                      int32_t *n_accept, int32_t *next_token, float *lse, void *ws, size_t ws_bytes,
                                      epq_stream_t stream) {
  if (!logits || !tokens || !parent || !path || !n_accept || !next_token) return EPQ_ERR_ARG;
  const size_t need = epq_verify_tree_workspace_bytes(n_seq, ntok, vocab);
  if (!need) return EPQ_ERR_SHAPE;
  VerifyParams p = {};
  const float temperature = opts ? opts->temperature : 1.0f;
  if (!(temperature >= 0.0f) || std::isinf(temperature)) return EPQ_ERR_ARG;
  p.greedy = temperature == 0.0f;
  if (!p.greedy && !u) return EPQ_ERR_ARG;
  p.ld = opts && opts->ld ? opts->ld : vocab;
  p.draft_ld = opts && opts->draft_ld ? opts->draft_ld : vocab;
  if (p.ld < vocab || p.draft_ld < vocab) return EPQ_ERR_SHAPE;
  if (!ws || ws_bytes < need) return EPQ_ERR_WORKSPACE;
  if (((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(opts ? opts->draft : nullptr)) & 3) ||
      !aligned16(ws))
    return EPQ_ERR_ALIGN;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  const int64_t rows = static_cast<int64_t>(n_seq) * ntok;
  p.logits = logits;
  p.draft = opts ? opts->draft : nullptr;
  p.u = u;
  p.tokens = tokens;
  p.parent = parent;
  p.n_tok = opts ? opts->n_tok : nullptr;
  p.vocab = static_cast<int>(vocab);
  p.n_seq = n_seq;
  p.ntok = ntok;
  p.splits = static_cast<int>(stats_splits(rows, vocab));
  // finite in float32 for the smallest temperatures too
  const double c = std::min(1.4426950408889634 / (p.greedy ? 1.0 : static_cast<double>(temperature)), 3.4e38);
  p.c_hi = static_cast<float>(c);
  p.c_lo = static_cast<float>(c - static_cast<double>(p.c_hi));
  p.inv_t = p.greedy ? 1.0f : static_cast<float>(1.0 / static_cast<double>(temperature));
  p.path = path;
  p.n_accept = n_accept;
  p.next_token = next_token;
  p.lse = lse;
  p.part_max = static_cast<float *>(ws);
  p.part_sum = p.part_max + rows * p.splits;
  p.part_arg = reinterpret_cast<int32_t *>(p.part_sum + rows * p.splits);
  for (int j = 0; j < 32; ++j) p.table[j] = static_cast<unsigned long long>(std::exp2(j / 32.0) * 4611686018427387904.0);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(p.splits, static_cast<unsigned>(rows));
  cudaError_t e = stats_chunk(rows, vocab) == 8192 ? launch_pdl(row_stats_kernel<8>, grid, dim3(kStatThreads), 0, s, p)
                                                   : launch_pdl(row_stats_kernel<2>, grid, dim3(kStatThreads), 0, s, p);
  if (e != cudaSuccess) return cuda_fail(e);
  const size_t smem = 12 * static_cast<size_t>(kWalkWarps) * walk_entries(p.vocab);
  static LaunchOnce once;
  e = once.prepare(dev.device, walk_kernel, kWalkThreads, 12 * static_cast<size_t>(kWalkWarps) * walk_entries(kMaxVocab),
                   true, nullptr);
  if (e != cudaSuccess) return cuda_fail(e);
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(static_cast<unsigned>(n_seq) * kWalkCluster);
  cfg.blockDim = dim3(kWalkThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kWalkCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, walk_kernel, p);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
