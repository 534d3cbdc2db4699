// dec_kv_extend, dec_kv_fork, dec_kv_release and dec_kv_compact: the pages of a
// paged key/value cache, counted and copied on the device.
//
// Each call that allocates or moves pages plans in one CTA (its work is a scan
// over refs, a few ints per page), which checks everything and changes nothing
// on an error, and carries the plan out in a second launch over the whole GPU.
// (extend has a second one for 8-bit pages, whose scales it clears.)
// All choices are by rank (the k-th page needed gets the k-th lowest free one),
// so results do not depend on the order in which threads run.
#include "common.cuh"
#include "kv.h"

using namespace tld;

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyPiece = kCopyThreads * 16 * kCopyUnroll;  // 16 KB

// Words of the scratch head.
enum { SC_OK = 0, SC_MOVES = 1, SC_LIVE = 2 };

// Exclusive prefix sum over the CTA's kPlanThreads threads; *total gets the sum.
__device__ int block_scan(int x, int* total) {
  __shared__ int warp_sums[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // the sums of the previous call have been read
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  int s = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  const int before = w ? __shfl_sync(0xffffffffu, s, w - 1) : 0;
  *total = __shfl_sync(0xffffffffu, s, 31);
  return before + incl - x;
}

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// A sequence's length, or -1 if it is not one the table can hold.
__device__ __forceinline__ int kv_len(const KvView& c, int s) {
  const int n = c.lens[s];
  return n >= 0 && n <= c.max_pages * c.page_rows ? n : -1;
}

// Calls f(page, k-th of its kind, k-th of its kind) ... for every page in order:
// kind(page) puts a page into neither, the first or the second of two kinds (0,
// 1, 2), and f(page, kind, rank) gets its rank among those of its kind.  Four
// pages a thread at a time; stops once `enough` of the first kind are found.
// The counts of both kinds are returned to every thread.
template <class Kind, class F>
__device__ int2 rank_pages(int n_pages, int enough, Kind kind, F f) {
  int2 found = make_int2(0, 0);
  for (int base = 0; base < n_pages && found.x < enough; base += 4 * kPlanThreads) {
    int kinds[4], mine = 0;  // counts of both kinds in 16 bits each (at most 4096)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = base + 4 * threadIdx.x + i;
      kinds[i] = p < n_pages ? kind(p) : 0;
      mine += kinds[i] == 1 ? 1 : kinds[i] == 2 ? 1 << 16 : 0;
    }
    int total;
    int at = block_scan(mine, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = base + 4 * threadIdx.x + i;
      if (p < n_pages) f(p, kinds[i], kinds[i] == 1 ? found.x + (at & 0xffff) : found.y + (at >> 16));
      at += kinds[i] == 1 ? 1 : kinds[i] == 2 ? 1 << 16 : 0;
    }
    found.x += total & 0xffff;
    found.y += total >> 16;
  }
  __syncthreads();
  return found;
}

// Lists the `need` lowest free pages in the scratch; false if there are fewer.
__device__ bool find_free(const KvView& c, int need) {
  int32_t* list = c.scratch + kKvScratchHead;
  return rank_pages(c.n_pages, need, [&](int p) { return c.refs[p] <= 0 ? 1 : 0; },
                    [&](int p, int kind, int rank) {
                      if (kind && rank < need && KV_IN_BOUNDS(c, rank >= 0 && rank < c.n_pages)) list[rank] = p;
                    }).x >= need;
}

// FORK: a = parents, b = children.  Otherwise extend: a = sequences, b = rows to add.
template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) kv_plan_alloc(KvView c, const int32_t* a, const int32_t* b, int n) {
  __shared__ uint32_t seen[65536 / 32];
  __shared__ int bad_bits;
  pdl_trigger();  // (nothing before the launch behind it waits for the end of this one)
  const int tid = threadIdx.x;
  int32_t* offsets = c.scratch + kv_scratch_offsets(c.n_pages, c.n_seqs);
  int32_t* moves = c.scratch + kv_scratch_moves(c.n_pages);
  for (int i = tid; i < (c.n_seqs + 31) / 32; i += kPlanThreads) seen[i] = 0;
  if (tid == 0) bad_bits = 0;
  __syncthreads();

  int total = 0;  // pages needed, at most n_pages + 1
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0, bad = 0;
    if (i < n) {
      const int s = a ? a[i] : i;
      const int x = b ? b[i] : 1;  // child, or rows to add
      if (s >= 0 && (!FORK || x >= 0)) {
        if (s >= c.n_seqs || (FORK ? x >= c.n_seqs : x < 0)) {
          bad = DEC_KV_BAD_INDEX;
        } else {
          const int mark = FORK ? x : s;
          if (atomicOr(&seen[mark >> 5], 1u << (mark & 31)) >> (mark & 31) & 1) bad = DEC_KV_BAD_LIST;
          const int len = kv_len(c, s);
          if (len < 0) {
            bad |= DEC_KV_BAD_INDEX;
          } else if (FORK) {
            if (c.lens[x] != 0) bad |= DEC_KV_BAD_LIST;
            need = len % c.page_rows != 0;
            if (need) {
              const int tail = c.table[(int64_t)s * c.max_pages + len / c.page_rows];
              if (tail < 0 || tail >= c.n_pages) bad |= DEC_KV_BAD_INDEX;
            }
          } else if (x > c.max_pages * c.page_rows - len) {
            bad |= DEC_KV_NO_PAGES;
          } else {
            need = div_up(len + x, c.page_rows) - div_up(len, c.page_rows);
          }
        }
      }
    }
    if (bad) {
      atomicOr(&bad_bits, bad);
      need = 0;
    }
    int sum;
    const int at = total + block_scan(min(need, c.n_pages + 1), &sum);
    if (i < n) offsets[i] = at;
    total = min(total + sum, c.n_pages + 1);
  }
  if (tid == 0) offsets[n] = total;
  __syncthreads();
  if (FORK) {
    // A parent that is also a child would be copied before or after it changes, and
    // pages that are none would be copied into the child's table: a warp per entry, or
    // 2^more of them where there are few entries.
    constexpr int kWarps = kPlanThreads / 32;
    const int more = max(__clz(n - 1) - __clz(kWarps - 1), 0);
    for (int unit = tid >> 5; unit >> more < n; unit += kWarps) {
      const int i = unit >> more, s = a[i], x = b[i];
      if (s < 0 || s >= c.n_seqs || x < 0) continue;
      const int32_t* row = c.table + (int64_t)s * c.max_pages;
      int most = -1;
#pragma unroll 16
      for (int at = (unit & ((1 << more) - 1)) * 32 + (tid & 31); at < c.max_pages; at += 32 << more)
        most = max(most, row[at]);
      const int bad = (seen[s >> 5] >> (s & 31) & 1 ? DEC_KV_BAD_LIST : 0) | (most >= c.n_pages ? DEC_KV_BAD_INDEX : 0);
      if (bad) atomicOr(&bad_bits, bad);
    }
    __syncthreads();
  }
  int bad = bad_bits;  // the same in every thread, as are total and find_free's answer
  if (!bad && (total > c.n_pages || !find_free(c, total))) bad = DEC_KV_NO_PAGES;
  if (bad) {
    if (tid == 0) {
      atomicOr(c.status, bad);
      c.scratch[SC_OK] = 0;
      c.scratch[SC_MOVES] = 0;
    }
    return;
  }

  const int32_t* list = c.scratch + kKvScratchHead;
  if (FORK) {
    for (int i = tid; i < n; i += kPlanThreads) {
      const int at = offsets[i];
      if (offsets[i + 1] > at) {
        const int s = a[i];
        if (!KV_IN_BOUNDS(c, at >= 0 && at < c.n_seqs && at < total && c.lens[s] / c.page_rows < c.max_pages)) continue;
        moves[2 * at] = c.table[(int64_t)s * c.max_pages + c.lens[s] / c.page_rows];
        moves[2 * at + 1] = list[at];
      }
    }
  } else {
    for (int k = tid; k < total; k += kPlanThreads) {  // page k belongs to the last entry starting at or before it
      int lo = 0, hi = n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (offsets[mid] <= k) lo = mid;
        else hi = mid;
      }
      const int s = a ? a[lo] : lo;
      const int place = div_up(c.lens[s], c.page_rows) + k - offsets[lo];
      if (!KV_IN_BOUNDS(c, k < c.n_pages && s >= 0 && s < c.n_seqs && place >= 0 && place < c.max_pages &&
                               list[k] >= 0 && list[k] < c.n_pages))
        continue;
      c.table[(int64_t)s * c.max_pages + place] = list[k];
      c.refs[list[k]] = 1;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kPlanThreads) {
      const int s = a ? a[i] : i;
      if (s >= 0) c.lens[s] += b ? b[i] : 1;
    }
  }
  if (tid == 0) {
    c.scratch[SC_OK] = 1;
    c.scratch[SC_MOVES] = total;
  }
}

// Ranks the live pages from `live` on against the free pages below it, renames
// them in refs and lists the copies.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_compact(KvView c) {
  pdl_trigger();
  const int tid = threadIdx.x;
  int32_t* name = c.scratch + kKvScratchHead;
  int32_t* moves = c.scratch + kv_scratch_moves(c.n_pages);
  const int all = 0x7fffffff;
  const int live = rank_pages(c.n_pages, all, [&](int p) { return c.refs[p] > 0 ? 1 : 0; }, [](int, int, int) {}).x;
  const int movers = rank_pages(
      c.n_pages, all,
      [&](int p) {
        const bool used = c.refs[p] > 0;
        return p < live ? (used ? 0 : 1) : (used ? 2 : 0);
      },
      [&](int p, int kind, int rank) {
        if (kind && KV_IN_BOUNDS(c, rank >= 0 && 2 * rank + 1 < c.n_pages + 2 * c.n_seqs))
          moves[2 * rank + (kind == 1)] = p;
        name[p] = kind == 0 && p < live ? p : -1;  // (those that move get theirs below)
      }).y;
  for (int k = tid; k < movers; k += kPlanThreads) {
    const int from = moves[2 * k], to = moves[2 * k + 1];
    if (!KV_IN_BOUNDS(c, from >= live && from < c.n_pages && to >= 0 && to < live)) continue;
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
    name[from] = to;
  }
  if (tid == 0) {
    c.scratch[SC_OK] = 1;
    c.scratch[SC_MOVES] = movers;
    c.scratch[SC_LIVE] = live;
  }
}

// 8-bit pages that a sequence has been given: scales of 0 in every layer.  A block that is
// not begun at its first row keeps its old scale where it is the larger one, and that of
// a page's last owner, or of memory that no one wrote, is none of its own.
__global__ void __launch_bounds__(kCopyThreads) kv_fresh(KvView c, int n_layers) {
  pdl_wait();
  const int32_t* list = c.scratch + kKvScratchHead;
  const uint32_t scales = (uint32_t)c.nkv * (c.page_rows / kBlockRows);  // of a page's K, or V
  const int64_t total = (int64_t)c.scratch[SC_MOVES] * n_layers * 2 * scales;
  for (int64_t e = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; e < total; e += (int64_t)gridDim.x * kCopyThreads) {
    const uint32_t i = (uint32_t)(e % scales);
    const int64_t rest = e / scales, page = rest / 2 / n_layers;
    const int layer = (int)(rest / 2 % n_layers), at = list[page];
    if (!KV_IN_BOUNDS(c, page < c.n_pages && at >= 0 && at < c.n_pages)) continue;
    uint8_t* half = c.pool + ((int64_t)layer * c.n_pages + at) * c.page_bytes + rest % 2 * c.half_bytes;
    reinterpret_cast<float*>(half + c.nkv * c.head_bytes)[i] = 0.f;
  }
}

// Carries out a plan: copies the listed pages in every layer; FORK: writes the
// children's table rows and counts; otherwise (compact) renames the pages in
// every table.
template <bool FORK>
__global__ void __launch_bounds__(kCopyThreads) kv_apply(KvView c, const int32_t* parents, const int32_t* children,
                                                         int n, int n_layers) {
  pdl_wait();
  if (!c.scratch[SC_OK]) return;
  const int64_t thread = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  const int64_t threads = (int64_t)gridDim.x * kCopyThreads;
  if (FORK) {
    const int32_t* offsets = c.scratch + kv_scratch_offsets(c.n_pages, c.n_seqs);
    const int32_t* list = c.scratch + kKvScratchHead;
    for (int64_t e = thread; e < (int64_t)n * c.max_pages; e += threads) {
      const int i = (int)(e / c.max_pages), at = (int)(e % c.max_pages);
      const int p = parents[i], ch = children[i];
      if (p < 0 || ch < 0) continue;
      const int len = c.lens[p];
      int page = c.table[(int64_t)p * c.max_pages + at];
      if (len % c.page_rows && at == len / c.page_rows) {
        page = list[offsets[i]];
        if (!KV_IN_BOUNDS(c, page >= 0 && page < c.n_pages)) continue;
        c.refs[page] = 1;
      } else if (page >= 0 && page < c.n_pages) {
        atomicAdd(c.refs + page, 1);
      }
      c.table[(int64_t)ch * c.max_pages + at] = page;
      if (at == 0) c.lens[ch] = len;
    }
  } else {
    const int32_t* name = c.scratch + kKvScratchHead;
    for (int64_t e = thread; e < (int64_t)c.n_seqs * c.max_pages; e += threads) {
      const int page = c.table[e];
      if (page < 0) continue;
      const int now = page < c.n_pages ? name[page] : -1;
      if (now < 0) atomicOr(c.status, DEC_KV_BAD_INDEX);
      else if (now != page) c.table[e] = now;
    }
  }
  // Pieces of kCopyPiece bytes of a page, in turn: 64 bytes a thread under way
  // (124 pages of four layers, 1.04 GB read and written: 172 us with the plan, 0.90 of
  // the copy rate).
  const int32_t* moves = c.scratch + kv_scratch_moves(c.n_pages);
  const uint32_t pieces = (uint32_t)((c.page_bytes + kCopyPiece - 1) / kCopyPiece);
  const int64_t total = (int64_t)c.scratch[SC_MOVES] * n_layers * pieces;
  for (int64_t e = blockIdx.x; e < total; e += gridDim.x) {
    const uint32_t piece = (uint32_t)(e % pieces);
    const int64_t rest = e / pieces;
    const int layer = (int)(rest % n_layers), m = (int)(rest / n_layers);
    if (!KV_IN_BOUNDS(c, moves[2 * m] >= 0 && moves[2 * m] < c.n_pages && moves[2 * m + 1] >= 0 &&
                             moves[2 * m + 1] < c.n_pages && layer < n_layers))
      continue;
    uint8_t* pages = c.pool + (int64_t)layer * c.n_pages * c.page_bytes;
    const int64_t at = (int64_t)piece * kCopyPiece + 16 * threadIdx.x;
    const uint8_t* from = pages + moves[2 * m] * c.page_bytes + at;
    uint8_t* to = pages + moves[2 * m + 1] * c.page_bytes + at;
    uint4 w[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (at + i * 16 * kCopyThreads < c.page_bytes) w[i] = __ldcs(reinterpret_cast<const uint4*>(from + i * 16 * kCopyThreads));
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (at + i * 16 * kCopyThreads < c.page_bytes) __stcs(reinterpret_cast<uint4*>(to + i * 16 * kCopyThreads), w[i]);
  }
}

// One CTA per list entry: takes the sequence's pages out of its table.
__global__ void __launch_bounds__(kCopyThreads) kv_release(KvView c, const int32_t* seqs, int window, int sinks) {
  const int s = seqs ? seqs[blockIdx.x] : blockIdx.x;
  if (s < 0) return;
  const int len = s < c.n_seqs ? kv_len(c, s) : -1;
  if (len < 0) {
    if (threadIdx.x == 0) atomicOr(c.status, DEC_KV_BAD_INDEX);
    return;
  }
  int first = 0, last = c.max_pages;
  if (window) {
    first = sinks / c.page_rows + (sinks % c.page_rows != 0);
    last = len > window ? (len - window) / c.page_rows : 0;
  }
  for (int i = first + threadIdx.x; i < last; i += kCopyThreads) {
    int32_t* entry = c.table + (int64_t)s * c.max_pages + i;
    if (*entry < 0) continue;
    const int page = atomicExch(entry, -1);  // a sequence listed twice gives each page back once
    if (page < 0) continue;
    if (page < c.n_pages) atomicSub(c.refs + page, 1);
    else atomicOr(c.status, DEC_KV_BAD_INDEX);
  }
  if (!window && threadIdx.x == 0) c.lens[s] = 0;
}

cudaLaunchConfig_t config(int64_t ctas, int threads, dec_stream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  return cfg;
}

// The launch that carries out a plan: it may begin before the plan's ends, and waits for it.
template <class... Args>
cudaError_t launch_after(void (*kernel)(Args...), int64_t ctas, dec_stream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = config(ctas, kCopyThreads, stream);
  cudaLaunchAttribute pdl = {};
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail_no_handle(DEC_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  return DEC_OK;
}

int launched(cudaError_t e) {
  return e == cudaSuccess ? DEC_OK : fail_no_handle(DEC_ERR_CUDA, "page kernel launch: %s", cudaGetErrorString(e));
}

int check_list(const dec_kv_cache* c, int n) {
  if (int rc = kv_check(c, true)) return rc;
  if (n < 0 || n > c->n_seqs) return fail_no_handle(DEC_ERR_ARG, "a list of %d of %d sequences", n, c->n_seqs);
  return DEC_OK;
}

}  // namespace

extern "C" int dec_kv_extend(const dec_kv_cache* c, const int32_t* seqs, const int32_t* n_new, int n,
                             dec_stream_t stream) {
  if (int rc = check_list(c, n)) return rc;
  if (n == 0) return DEC_OK;
  const bool blocks = c->format == DEC_KV_Q8T16;
  int sms = 0;
  if (blocks)
    if (int rc = sm_count(&sms)) return rc;
  const KvView v = kv_view(*c, 0);
  const cudaLaunchConfig_t plan = config(1, kPlanThreads, stream);
  const int rc = launched(cudaLaunchKernelEx(&plan, kv_plan_alloc<false>, v, seqs, n_new, n));
  return rc || !blocks ? rc : launched(launch_after(kv_fresh, 2 * sms, stream, v, (int)c->n_layers));
}

extern "C" int dec_kv_fork(const dec_kv_cache* c, const int32_t* parents, const int32_t* children, int n,
                           dec_stream_t stream) {
  if (int rc = check_list(c, n)) return rc;
  if (n == 0) return DEC_OK;
  if (!parents || !children) return fail_no_handle(DEC_ERR_ARG, "parents or children is NULL");
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  const KvView v = kv_view(*c, 0);
  const cudaLaunchConfig_t plan = config(1, kPlanThreads, stream);
  if (int rc = launched(cudaLaunchKernelEx(&plan, kv_plan_alloc<true>, v, parents, children, n))) return rc;
  return launched(launch_after(kv_apply<true>, 8 * sms, stream, v, parents, children, n, (int)c->n_layers));
}

extern "C" int dec_kv_release(const dec_kv_cache* c, const int32_t* seqs, int n, int window, int sinks,
                              dec_stream_t stream) {
  if (int rc = check_list(c, n)) return rc;
  if (window < 0 || sinks < 0) return fail_no_handle(DEC_ERR_ARG, "window %d, sinks %d", window, sinks);
  if (n == 0) return DEC_OK;
  const cudaLaunchConfig_t cfg = config(n, kCopyThreads, stream);
  return launched(cudaLaunchKernelEx(&cfg, kv_release, kv_view(*c, 0), seqs, window, sinks));
}

extern "C" int dec_kv_compact(const dec_kv_cache* c, dec_stream_t stream) {
  if (int rc = kv_check(c, true)) return rc;
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  const KvView v = kv_view(*c, 0);
  const cudaLaunchConfig_t plan = config(1, kPlanThreads, stream);
  if (int rc = launched(cudaLaunchKernelEx(&plan, kv_plan_compact, v))) return rc;
  return launched(launch_after(kv_apply<false>, 8 * sms, stream, v, (const int32_t*)nullptr, (const int32_t*)nullptr, 0,
                               (int)c->n_layers));
}
