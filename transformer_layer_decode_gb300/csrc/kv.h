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
  int32_t* owners;  // 8-bit pages: [n_pages][page_rows] of the layer (kv_write8)
  int64_t page_bytes;
  int64_t half_bytes;  // of K (or V) in a page
  int64_t head_bytes;  // of K (or V) of one head in a page (8 bits: without the scales)
  int n_pages, n_seqs, max_pages, page_rows, nkv;
};

// The formats as the kernels' template parameter.
enum KvFormat { KV_BF16 = DEC_KV_BF16, KV_Q4 = DEC_KV_Q4B32, KV_Q8 = DEC_KV_Q8T16 };

// Bytes of one row of K or V of one head, scales included (8 bits: without).
__host__ __device__ inline int kv_row_bytes(int head_dim, int format) {
  return format == KV_Q8 ? head_dim : format == KV_Q4 ? head_dim / 2 + head_dim / 16 : 2 * head_dim;
}

constexpr int kBlockRows = 16;  // rows of a block of 8-bit pages

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

#ifdef __CUDACC__
// Where row t of a call's lists lies: its page's first byte (null: skipped; noted where
// an index was bad), its row in it, its sequence and position.
struct KvPlace {
  uint8_t* page;
  int row, seq, pos;
};
__device__ __forceinline__ KvPlace kv_place(const KvView& c, const int32_t* seqs, const int32_t* positions, int64_t t, int n) {
  KvPlace at{nullptr, 0, -1, 0};
  const int s = t < n ? (seqs ? seqs[t] : (int)t) : -1;
  if (s < 0) return at;
  int page = -1;
  if (s < c.n_seqs) {
    const int pos = positions ? positions[t] : c.lens[s] - 1;
    if (pos >= 0 && pos < c.max_pages * c.page_rows) {
      page = c.table[(int64_t)s * c.max_pages + pos / c.page_rows];
      at.row = pos % c.page_rows, at.seq = s, at.pos = pos;
    }
  }
  if (page >= 0 && page < c.n_pages) at.page = c.pool + page * c.page_bytes;
  else atomicOr(c.status, DEC_KV_BAD_INDEX);
  return at;
}

#endif

// A launch that is set up while the kernel before it runs (one that calls pdl_trigger) or
// ends.  Each of its threads calls pdl_wait before its first access to global memory:
// only behind it is what earlier kernels wrote there to be seen, and a kernel of which a
// block left without waiting could be over before the one before it.
struct BehindLast {
  cudaLaunchAttribute pdl = {};
  explicit BehindLast(cudaLaunchConfig_t* cfg) {
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = &pdl;
    cfg->numAttrs = 1;
  }
  BehindLast(const BehindLast&) = delete;
};

struct RopeRows;
// dec_kv_append to 8-bit pages (and dec_kv_append_rotated, with q).
cudaError_t kv_write8(const KvView& c, int head_dim, bool f32, const void* k, const void* v, int64_t stride,
                      const int32_t* seqs, const int32_t* positions, int n, const RopeRows* q, cudaStream_t s);

// Checks a cache (its pointers too, with `memory`); DEC_OK or the error, recorded.
int kv_check(const dec_kv_cache* c, bool memory);
KvView kv_view(const dec_kv_cache& c, int layer);

// Whether rows of wa bytes at a + i * sa and of wb bytes at b + i * sb (i < n) share a
// byte (where sa and sb differ: whether what they span does).
inline bool kv_rows_overlap(uintptr_t a, int64_t sa, int64_t wa, uintptr_t b, int64_t sb, int64_t wb, int n) {
  if (a + (n - 1) * sa + wa <= b || b + (n - 1) * sb + wb <= a) return false;
  if (sa != sb) return true;
  const int64_t d = (int64_t)(a > b ? a - b : b - a) % sa;  // how far behind the one that begins first the other does
  return d < (a > b ? wb : wa) || d > sa - (a > b ? wa : wb);
}
inline bool kv_rows_overlap(uintptr_t a, int64_t sa, uintptr_t b, int64_t sb, int64_t width, int n) {
  return kv_rows_overlap(a, sa, width, b, sb, width, n);
}

}  // namespace tld
