// The paged Q8_0 cache as the kernels see it (epq_pages): host checks, device
// addressing.
#pragma once

#include <atomic>

#include "common.cuh"

namespace epq {

constexpr int kMaxSeq = 256;      // sequences of one cache
constexpr int kMaxTree = 64;      // drafted tokens of one sequence (bits of a mask word)

struct PagesView {
  uint8_t *pool;
  int32_t *table, *length, *refs;
  int32_t *work;
  int n_layers, n_pages, n_kv, D, P, n_seq, max_pages;
  int row;             // bytes of one cached row
  int64_t head_bytes;  // K and V planes of one (page, head)
  int64_t page_bytes;
  int64_t layer_bytes;
};

// Sizes only (no pointer is looked at).
inline bool pages_sizes_ok(const epq_pages *p) {
  return p && p->n_layers >= 1 && p->n_pages >= 1 && p->n_kv_heads >= 1 && p->n_kv_heads <= 256 &&
         epq_kv_row_bytes(p->head_dim) > 0 &&
         (p->page_size == 16 || p->page_size == 32 || p->page_size == 64 || p->page_size == 128) && p->n_seq >= 1 &&
         p->n_seq <= kMaxSeq && p->max_pages >= 1 &&
         static_cast<int64_t>(p->max_pages) * p->page_size <= (int64_t(1) << 30) && p->n_pages <= (1 << 28) &&
         p->n_layers <= (1 << 16);
}

inline epq_status pages_view(const epq_pages *p, PagesView *v) {
  if (!p) return EPQ_ERR_ARG;
  if (!pages_sizes_ok(p)) return EPQ_ERR_SHAPE;
  if (!p->pool || !p->table || !p->length || !p->refs || !p->work) return EPQ_ERR_ARG;
  if (!aligned16(p->pool) || !aligned16(p->table) || !aligned16(p->length) || !aligned16(p->refs) ||
      !aligned16(p->work))
    return EPQ_ERR_ALIGN;
  v->pool = static_cast<uint8_t *>(p->pool);
  v->table = p->table;
  v->length = p->length;
  v->refs = p->refs;
  v->work = static_cast<int32_t *>(p->work);
  v->n_layers = p->n_layers;
  v->n_pages = p->n_pages;
  v->n_kv = p->n_kv_heads;
  v->D = p->head_dim;
  v->P = p->page_size;
  v->n_seq = p->n_seq;
  v->max_pages = p->max_pages;
  v->row = static_cast<int>(epq_kv_row_bytes(p->head_dim));
  v->head_bytes = 2ll * p->page_size * v->row;
  v->page_bytes = v->head_bytes * p->n_kv_heads;
  v->layer_bytes = v->page_bytes * p->n_pages;
  return EPQ_OK;
}

// What a kernel's launch needs to know or set once per device: its dynamic
// shared-memory limit (and the opt-in to clusters of more than 8 CTAs), and
// how many of its CTAs fit an SM.  A value is looked up once and kept.
class LaunchOnce {
 public:
  template <typename K>
  cudaError_t prepare(int device, K kernel, int threads, size_t smem, bool large_cluster, int *per_sm) {
    std::atomic<int> &slot = known_[device];
    int n = slot.load(std::memory_order_acquire);
    if (n == 0) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e == cudaSuccess && large_cluster)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
      if (e != cudaSuccess) return e;
      n = n > 0 ? n : 1;
      slot.store(n, std::memory_order_release);
    }
    if (per_sm) *per_sm = n;
    return cudaSuccess;
  }

 private:
  std::atomic<int> known_[64] = {};  // current_device admits no more devices
};

#ifdef __CUDACC__
// Committed length of sequence s, held to what its table can address.
__device__ __forceinline__ int seq_length(const PagesView &v, int s) {
  return min(max(v.length[s], 0), v.max_pages * v.P);
}

// Page j of sequence s, or -1 when there is none (or no such page).
__device__ __forceinline__ int seq_page(const PagesView &v, int s, int j) {
  if (j < 0 || j >= v.max_pages) return -1;
  const int id = v.table[static_cast<int64_t>(s) * v.max_pages + j];
  return id >= 0 && id < v.n_pages ? id : -1;
}

// Row `slot` of plane c (0 keys, 1 values) of a page's head.
__device__ __forceinline__ uint8_t *page_row(const PagesView &v, int layer, int page, int head, int c, int slot) {
  return v.pool + layer * v.layer_bytes + page * v.page_bytes + head * v.head_bytes +
         static_cast<int64_t>(c * v.P + slot) * v.row;
}
#endif

}  // namespace epq
