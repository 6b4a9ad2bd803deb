// Pages of the paged Q8_0 cache: freeing, sharing, allocation with copy on
// write, and moving accepted rows together (epq_pages_*).
//
// The state is three integer arrays: table (a sequence's page ids), length
// (its committed positions) and refs (holders per page; 0 = free).  There is
// no free list: a free page is one with refs 0, and allocation takes the
// lowest such ids, so releasing is a decrement that needs no order and the
// result of every call is a function of the state alone.
#include <algorithm>

#include "pages.cuh"

namespace epq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 128;

// Layout of epq_pages.work (int32): 16 words of which the first counts the
// CTAs of a compact call that have read the lengths; the copies that reserve
// planned (source page, destination page, rows); the free ids that it found.
__host__ __device__ inline int work_ints(int n_seq, int n_pages) { return 16 + 3 * n_seq + n_pages; }

// ------------------------------------------------------------------ truncate
// One CTA per sequence; the only shared writes are the decrements.
__global__ void __launch_bounds__(256) truncate_kernel(const __grid_constant__ PagesView v,
                                                       const int32_t *__restrict__ new_length) {
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.x;
  const int want = new_length[s];
  const int len = min(seq_length(v, s), max(want, 0));
  __syncthreads();  // every thread has read the length that thread 0 replaces
  if (want < 0) return;
  int32_t *row = v.table + static_cast<int64_t>(s) * v.max_pages;
  for (int j = (len + v.P - 1) / v.P + threadIdx.x; j < v.max_pages; j += blockDim.x) {
    const int id = row[j];
    if (id >= 0 && id < v.n_pages) atomicSub(&v.refs[id], 1);
    row[j] = -1;
  }
  if (threadIdx.x == 0) v.length[s] = len;
}

// ------------------------------------------------------------------ fork
// One CTA per entry.  An entry reads only sequences that no entry of the call
// writes (a source that is also a destination is refused), so the CTAs are
// independent.
__global__ void __launch_bounds__(128) fork_kernel(const __grid_constant__ PagesView v, const int32_t *__restrict__ src,
                                                   const int32_t *__restrict__ dst, int n, int32_t *status) {
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x;
  const int a = src[i], b = dst[i];
  int bad = a < 0 || a >= v.n_seq || b < 0 || b >= v.n_seq || a == b;
  for (int k = threadIdx.x; k < n; k += blockDim.x) bad |= dst[k] == a || (k < i && dst[k] == b);
  if (!bad) bad = v.length[b] != 0 || v.table[static_cast<int64_t>(b) * v.max_pages] >= 0;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0 && status) status[i] = bad ? 1 : 0;
  if (bad) return;
  const int len = seq_length(v, a);
  const int32_t *from = v.table + static_cast<int64_t>(a) * v.max_pages;
  int32_t *to = v.table + static_cast<int64_t>(b) * v.max_pages;
  for (int j = threadIdx.x; j < (len + v.P - 1) / v.P; j += blockDim.x) {
    const int id = from[j];
    to[j] = id;
    if (id >= 0 && id < v.n_pages) atomicAdd(&v.refs[id], 1);
  }
  if (threadIdx.x == 0) v.length[b] = len;
}

// ------------------------------------------------------------------ reserve
// Inclusive sum over the CTA (1024 threads).
__device__ __forceinline__ long long block_scan(long long x, long long *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long base = 0;
  for (int w = 0; w < warp; ++w) base += warp_sums[w];
  return base + x;
}

// One CTA: thread s works out what sequence s needs; the free ids are found
// in rising order; tables and refs are brought up to date and the planned
// copies (source, destination, rows) left in `work` for the copy kernel.
__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(const __grid_constant__ PagesView v,
                                                                    const int32_t *__restrict__ extra,
                                                                    int32_t *__restrict__ status) {
  __shared__ long long warp_sums[32];
  __shared__ int held[kMaxSeq];        // partly filled last page of an active sequence, or -1
  __shared__ long long upto[kMaxSeq];  // pages needed up to and with sequence s
  __shared__ int found_all;
  pdl_launch_dependents();
  pdl_wait();
  const int s = threadIdx.x;
  int32_t *plan = v.work + 16;
  int32_t *ids = plan + 3 * v.n_seq;
  int first = 0, last = 0, len = 0, ex = 0, mine = -1, copies = 0;
  bool active = false, fits = true;
  if (s < v.n_seq) {
    len = seq_length(v, s);
    ex = extra[s];
    const long long end = (static_cast<long long>(len) + max(ex, 0) + v.P - 1) / v.P;
    fits = end <= v.max_pages;
    active = ex > 0 && fits;
    first = len / v.P;
    last = active ? static_cast<int>(end) : first;
    if (active && len % v.P) mine = seq_page(v, s, first);
    held[s] = mine;
  }
  __syncthreads();
  long long need = 0;
  if (active) {
    if (mine >= 0) {
      int rank = 0;
      for (int k = 0; k < s; ++k) rank += held[k] == mine;
      copies = v.refs[mine] - rank > 1;
    }
    need = copies;
    for (int j = first; j < last; ++j) need += seq_page(v, s, j) < 0;
  }
  const long long end = block_scan(need, warp_sums);
  if (s < v.n_seq) upto[s] = end;
  __syncthreads();
  const long long wanted = upto[v.n_seq - 1];
  // the lowest `wanted` free ids
  long long found = 0;
  for (int base = 0; base < v.n_pages && found < wanted; base += kPlanThreads) {
    const int id = base + threadIdx.x;
    const bool is_free = id < v.n_pages && v.refs[id] == 0;
    const long long at = found + block_scan(is_free ? 1 : 0, warp_sums);
    if (is_free && at <= wanted) ids[at - 1] = id;
    if (threadIdx.x == kPlanThreads - 1) found_all = static_cast<int>(at < wanted ? at : wanted);
    __syncthreads();
    found = found_all;
    __syncthreads();
  }
  __syncthreads();  // the ids are visible to the CTA
  if (s < v.n_seq) {
    const bool ok = end <= found;
    if (!active || !ok) copies = 0;
    if (active && ok) {
      int32_t *row = v.table + static_cast<int64_t>(s) * v.max_pages;
      long long at = end - need;
      for (int j = first; j < last; ++j) {
        if (!(seq_page(v, s, j) < 0 || (copies && j == first))) continue;
        const int id = ids[at++];
        row[j] = id;
        v.refs[id] = 1;
      }
      if (copies) atomicSub(&v.refs[mine], 1);
    }
    plan[3 * s] = mine;
    plan[3 * s + 1] = copies ? seq_page(v, s, first) : -1;
    plan[3 * s + 2] = copies ? len % v.P : 0;
    if (status) status[s] = ex <= 0 ? 0 : !fits ? 2 : ok ? 0 : 1;
  }
}

// Grid (layers * heads * 2 planes, groups of sequences): the committed rows of
// the copied pages.  The planes go through shared memory with bulk copies: one
// load for all branches of a page that follow one another, one store each.
// Bound by DRAM writes: 508 MB of copies of 22 MB take 89 us, 5.9 TB/s (0.88
// of the copy bandwidth); a CTA of 128 threads per copy, which read the page
// again for each, took 96 us.
__global__ void __launch_bounds__(32) reserve_copy_kernel(const __grid_constant__ PagesView v, int per_cta,
                                                          unsigned *err) {
  extern __shared__ __align__(128) uint8_t plane[];  // [page_size][row]
  __shared__ uint64_t bar;
  const int lane = threadIdx.x;
  if (lane == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x & 1, h = (blockIdx.x >> 1) % v.n_kv, layer = (blockIdx.x >> 1) / v.n_kv;
  const int s0 = blockIdx.y * per_cta, s1 = min(s0 + per_cta, v.n_seq);
  int held = -1, held_rows = 0;
  uint32_t loads = 0;
  for (int s = s0; s < s1; ++s) {
    const int32_t *plan = v.work + 16 + 3 * s;
    const int from = plan[0], to = plan[1], rows = plan[2];
    if (rows == 0) continue;
    const uint8_t *a = page_row(v, layer, from, h, c, 0);
    uint8_t *b = page_row(v, layer, to, h, c, 0);
    const uint32_t bytes = static_cast<uint32_t>(rows) * v.row;  // a multiple of 8; the plane starts on 16
    if (from != held || rows != held_rows) {
      if (lane == 0) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the stores have read the plane
        mbar_arrive_expect_tx(&bar, bytes & ~15u);
        bulk_g2s(plane, a, bytes & ~15u, &bar);
      }
      if (!warp_wait(&bar, loads & 1, err, DEVERR_FULL_WAIT, loads)) {
        warp_wait(&bar, loads & 1, err, DEVERR_DRAIN_WAIT, loads);
        break;
      }
      ++loads;
      held = from;
      held_rows = rows;
    }
    if (lane == 0) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                       static_cast<uint64_t>(__cvta_generic_to_global(b))),
                   "r"(smem_addr(plane)), "r"(bytes & ~15u)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    if ((bytes & 8) && lane == 1)
      *reinterpret_cast<uint2 *>(b + bytes - 8) = *reinterpret_cast<const uint2 *>(a + bytes - 8);
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------ compact
// Grid (CTAs over the units, sequences); a unit is one (layer, head, plane).
// Where a sequence's rows come from and go to is the same in every unit, so a
// CTA works it out once, and its warps take units.  A warp reads some rows into
// registers before it writes them: entry i comes from path[i] >= i, so the
// rows of later entries are never written before they are read.  The words'
// addresses are worked out once per batch of rows, ahead of the loop over the
// units.  24 sequences x 1280 units, 28 MB read: 17 us (21 us with the
// addresses worked out in every unit; a CTA per unit and sequence: 37 us).
constexpr int kMoveWords = 9;  // 8-byte words of a lane: 16 rows of 128 elements, 8 of 256

__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const __grid_constant__ PagesView v,
                                                               const int32_t *__restrict__ path,
                                                               const int32_t *__restrict__ n_keep, int ntok,
                                                               unsigned *err) {
  __shared__ long long from[kMaxTree], to[kMaxTree];  // byte offsets within a unit's head of a layer; -1: nothing moves
  __shared__ int moves, last;
  pdl_launch_dependents();
  pdl_wait();
  const int s = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) moves = 0;
  const int len = seq_length(v, s);
  const int n = min(max(n_keep[s], 0), ntok);
  __syncthreads();  // every thread has the length
  if (tid == 0) {
    // the last CTA to have read its sequence's length brings all lengths up to date
    __threadfence();
    last = atomicAdd(reinterpret_cast<unsigned *>(v.work), 1u) == gridDim.x * gridDim.y - 1;
  }
  if (tid < n) {
    const int p = path[s * ntok + tid];
    from[tid] = -1;
    if (p > tid && p < ntok) {
      const int a = seq_page(v, s, (len + p) / v.P), b = seq_page(v, s, (len + tid) / v.P);
      if (a >= 0 && b >= 0) {
        from[tid] = a * v.page_bytes + static_cast<long long>((len + p) % v.P) * v.row;
        to[tid] = b * v.page_bytes + static_cast<long long>((len + tid) % v.P) * v.row;
        moves = 1;
      } else {
        record_error(err, DEVERR_NO_PAGE, static_cast<unsigned>(s));
      }
    }
  }
  __syncthreads();
  if (last) {
    __threadfence();
    for (int k = tid; k < v.n_seq; k += kCopyThreads)
      v.length[k] = min(seq_length(v, k) + min(max(n_keep[k], 0), ntok), v.max_pages * v.P);
    if (tid == 0) v.work[0] = 0;
  }
  if (!moves) return;
  const int words = v.row / 8, batch = kMoveWords * 32 / words;
  const int units = v.n_layers * v.n_kv * 2, warps = gridDim.x * (kCopyThreads / 32);
  for (int i0 = 0; i0 < n; i0 += batch) {
    // where the lane's words come from and go to, in every unit
    const int all = min(batch, n - i0) * words;
    long long src[kMoveWords], dst[kMoveWords];
#pragma unroll
    for (int k = 0; k < kMoveWords; ++k) {
      const int x = 32 * k + lane, i = min(x, all - 1) / words;
      const bool moved = x < all && from[i0 + i] >= 0;
      src[k] = moved ? from[i0 + i] + 8 * (x - i * words) : -1;
      dst[k] = to[i0 + i] + 8 * (x - i * words);
    }
    for (int unit = blockIdx.x * (kCopyThreads / 32) + (tid >> 5); unit < units; unit += warps) {
      const int c = unit & 1, h = (unit >> 1) % v.n_kv, layer = (unit >> 1) / v.n_kv;
      uint8_t *base = page_row(v, layer, 0, h, c, 0);
      uint2 x[kMoveWords];
#pragma unroll
      for (int k = 0; k < kMoveWords; ++k)
        if (src[k] >= 0) x[k] = *reinterpret_cast<const uint2 *>(base + src[k]);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kMoveWords; ++k)
        if (src[k] >= 0) *reinterpret_cast<uint2 *>(base + dst[k]) = x[k];
    }
  }
}

bool device_ok() {
  DeviceInfo dev;
  return current_device(&dev) && dev.major * 10 + dev.minor >= 100;
}

}  // namespace
}  // namespace epq

using namespace epq;

extern "C" size_t epq_pages_work_bytes(const epq_pages *pages) {
  if (!pages_sizes_ok(pages)) return 0;
  return 4 * static_cast<size_t>(work_ints(pages->n_seq, pages->n_pages));
}

extern "C" epq_status epq_pages_truncate(const epq_pages *pages, const int32_t *new_length, epq_stream_t stream) {
  PagesView v;
  const epq_status st = pages_view(pages, &v);
  if (st != EPQ_OK) return st;
  if (!new_length) return EPQ_ERR_ARG;
  if (!device_ok()) return EPQ_ERR_DEVICE;
  const cudaError_t e = launch_pdl(truncate_kernel, dim3(v.n_seq), dim3(256), 0,
                                   reinterpret_cast<cudaStream_t>(stream), v, new_length);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}

extern "C" epq_status epq_pages_fork(const epq_pages *pages, const int32_t *src, const int32_t *dst, int n,
                                     int32_t *status, epq_stream_t stream) {
  PagesView v;
  const epq_status st = pages_view(pages, &v);
  if (st != EPQ_OK) return st;
  if (!src || !dst) return EPQ_ERR_ARG;
  if (n < 1 || n > kMaxSeq) return EPQ_ERR_SHAPE;
  if (!device_ok()) return EPQ_ERR_DEVICE;
  const cudaError_t e = launch_pdl(fork_kernel, dim3(n), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), v, src,
                                   dst, n, status);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}

extern "C" epq_status epq_pages_reserve(const epq_pages *pages, const int32_t *extra, int32_t *status,
                                        epq_stream_t stream) {
  PagesView v;
  const epq_status st = pages_view(pages, &v);
  if (st != EPQ_OK) return st;
  if (!extra || !status) return EPQ_ERR_ARG;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  unsigned *err = device_error_slot();
  if (!err) return EPQ_ERR_DEVICE;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(reserve_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, v, extra, status);
  if (e == cudaSuccess) {  // also for one sequence: another cache over the pool may hold its page
    // all branches in one CTA, unless that leaves SMs idle
    const int units = v.n_layers * v.n_kv * 2;
    const int groups = std::min(v.n_seq, std::max(1, 8 * dev.sm_count / units));
    const int per_cta = (v.n_seq + groups - 1) / groups;
    e = launch_pdl(reserve_copy_kernel, dim3(units, (v.n_seq + per_cta - 1) / per_cta), dim3(32),
                   static_cast<size_t>(v.P) * v.row, s, v, per_cta, err);
  }
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}

extern "C" epq_status epq_pages_compact(const epq_pages *pages, const int32_t *path, const int32_t *n_keep, int ntok,
                                        epq_stream_t stream) {
  PagesView v;
  const epq_status st = pages_view(pages, &v);
  if (st != EPQ_OK) return st;
  if (!path || !n_keep) return EPQ_ERR_ARG;
  if (ntok < 1 || ntok > kMaxTree) return EPQ_ERR_SHAPE;
  DeviceInfo dev;
  if (!current_device(&dev) || dev.major * 10 + dev.minor < 100) return EPQ_ERR_DEVICE;
  unsigned *err = device_error_slot();
  if (!err) return EPQ_ERR_DEVICE;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // enough warps for all units, but no more than a few CTAs per SM in all
  const int units = v.n_layers * v.n_kv * 2, warps = kCopyThreads / 32;
  const int x = std::max(1, std::min((units + warps - 1) / warps, 8 * dev.sm_count / v.n_seq));
  const cudaError_t e = launch_pdl(compact_kernel, dim3(x, v.n_seq), dim3(kCopyThreads), 0, s, v, path, n_keep, ntok, err);
  return e == cudaSuccess ? EPQ_OK : cuda_fail(e);
}
