// The paged key/value cache of many sequences: layout and the view its kernels take.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dec.h"

namespace tld {

// Records a message for dec_last_error(NULL) and returns `code`.
int fail_no_handle(int code, const char* fmt, ...) noexcept;

// One layer of a cache, as a kernel argument.
struct KvView {
  uint8_t* pool;  // the layer's pages
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int32_t* status;
  int32_t* scratch;
  int64_t page_bytes;
  int64_t half_bytes;  // of K (or V) in a page
  int64_t head_bytes;  // of K (or V) of one head in a page
  int n_pages, n_seqs, max_pages, page_rows, nkv;
};

// Bytes of one row of K or V of one head, scales included.
__host__ __device__ inline int kv_row_bytes(int head_dim, bool q4) {
  return q4 ? head_dim / 2 + head_dim / 16 : 2 * head_dim;
}

// The scratch of extend, fork and compact, in ints: a few words, the new names
// of pages (compact) or the free pages found (extend, fork), the page copies
// (source, destination), and where each list entry's pages start.
constexpr int kKvScratchHead = 32;
// Of the head's words: the source line of a check that failed (debug build), and
// beside it the status as dec_kv_status found it.
constexpr int kKvScratchLine = kKvScratchHead - 2, kKvScratchStatus = kKvScratchHead - 1;
__host__ __device__ inline int64_t kv_scratch_moves(int64_t n_pages) { return kKvScratchHead + n_pages; }
__host__ __device__ inline int64_t kv_scratch_offsets(int64_t n_pages, int64_t n_seqs) {
  return kv_scratch_moves(n_pages) + n_pages + 2 * n_seqs;
}
__host__ __device__ inline int64_t kv_scratch_ints(int64_t n_pages, int64_t n_seqs) {
  return kv_scratch_offsets(n_pages, n_seqs) + n_seqs + 1;
}

// Index checks of the debug build (TLD_DEBUG_CHECKS): one that fails sets
// DEC_KV_BAD_BOUNDS, notes its source line and is false, and the caller skips the
// access.  Release builds compile every check to true.
#ifdef TLD_DEBUG_CHECKS
__device__ __noinline__ inline bool kv_bounds_failed(const KvView& c, int line) {
  atomicExch(c.scratch + kKvScratchLine, line);
  atomicOr(c.status, DEC_KV_BAD_BOUNDS);
  return false;
}
#define KV_IN_BOUNDS(c, cond) ((cond) ? true : ::tld::kv_bounds_failed((c), __LINE__))
#else
#define KV_IN_BOUNDS(c, cond) true
#endif

// Checks a cache (its pointers too, with `memory`); DEC_OK or the error, recorded.
int kv_check(const dec_kv_cache* c, bool memory);
KvView kv_view(const dec_kv_cache& c, int layer);

// Whether rows of `width` bytes at a + i * sa and at b + i * sb (i < n) share a byte
// (where sa and sb differ: whether what they span does).
inline bool kv_rows_overlap(uintptr_t a, int64_t sa, uintptr_t b, int64_t sb, int64_t width, int n) {
  if (a + (n - 1) * sa + width <= b || b + (n - 1) * sb + width <= a) return false;
  if (sa != sb) return true;
  const int64_t d = (int64_t)(a > b ? a - b : b - a) % sa;
  return d < width || d > sa - width;
}

}  // namespace tld
