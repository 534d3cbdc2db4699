// dec_kv_attention: attention of one query per sequence over a paged key/value
// cache, bf16 or in 4-bit blocks, with a sliding window and first rows that
// stay visible.
#include <cmath>

#include "common.cuh"
#include "kv.h"

using namespace tld;

namespace {

constexpr int kSimpleThreads = 128;

struct KvAttnParams {
  KvView c;
  const void* q;
  void* o;
  int64_t q_stride, o_stride;
  const int32_t* seqs;
  int n, nq, window, sinks;
  float scale;
};

// Value e of a row of K or V of one head.
template <int D, bool Q4>
__device__ __forceinline__ float kv_value(const KvView& c, const uint8_t* head, int row, int e) {
  if constexpr (!Q4) {
    return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(head)[row * D + e] << 16);
  } else {
    constexpr int NB = D / 32;
    const int b = e / 32, nib = ((e % 32) / 4 * NB + b) * 4 + e % 4;
    const int byte = head[(int64_t)row * (D / 2) + nib / 2];
    const float s = __half2float(reinterpret_cast<const __half*>(head + (int64_t)c.page_rows * (D / 2))[row * NB + b]);
    return (float)((byte >> (4 * (nib & 1)) & 15) - 8) * s;
  }
}

// One CTA per (query head, query): chunks of 128 visible rows, a thread per
// row for the scores, a thread per dimension for the sums.
template <int D, bool Q4, class T>
__global__ void __launch_bounds__(kSimpleThreads) kv_attn_simple(KvAttnParams p) {
  __shared__ float q_s[D], w_s[kSimpleThreads], red[kSimpleThreads / 32];
  __shared__ const uint8_t* base_s[kSimpleThreads];
  __shared__ int row_s[kSimpleThreads];
  const KvView& c = p.c;
  const int tid = threadIdx.x, h = blockIdx.x, r = blockIdx.y;
  const int s = p.seqs ? p.seqs[r] : r;
  if (s < 0) return;
  const int len = s < c.n_seqs ? c.lens[s] : -1;
  if (len < 0 || len > c.max_pages * c.page_rows) {
    if (tid == 0) atomicOr(c.status, DEC_KV_BAD_INDEX);
    return;
  }
  const int lo = p.window ? max(len - p.window, 0) : 0, first = min(p.sinks, lo), count = first + len - lo;
  const int head = h / (p.nq / c.nkv);
  const T* q = static_cast<const T*>(p.q) + r * p.q_stride + (int64_t)h * D;
  for (int e = tid; e < D; e += kSimpleThreads) {
    if constexpr (sizeof(T) == 4) q_s[e] = q[e];
    else q_s[e] = __uint_as_float((uint32_t)q[e] << 16);
  }
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = 0; j0 < count; j0 += kSimpleThreads) {
    __syncthreads();
    const int j = j0 + tid;
    const uint8_t* base = nullptr;
    int row = 0;
    float score = -INFINITY;
    if (j < count) {
      const int pos = j < first ? j : lo + j - first;
      const int page = c.table[(int64_t)s * c.max_pages + pos / c.page_rows];
      row = pos % c.page_rows;
      if (page >= 0 && page < c.n_pages) {
        base = c.pool + page * c.page_bytes + head * c.head_bytes;
        float dot = 0.f;
        for (int e = 0; e < D; ++e) dot = fmaf(q_s[e], kv_value<D, Q4>(c, base, row, e), dot);
        score = dot * p.scale;
      } else {
        atomicOr(c.status, DEC_KV_BAD_INDEX);
      }
    }
    float top = warp_max(score);
    if ((tid & 31) == 0) red[tid >> 5] = top;
    base_s[tid] = base;
    row_s[tid] = row;
    __syncthreads();
    for (int w = 0; w < kSimpleThreads / 32; ++w) top = fmaxf(top, red[w]);
    const float m_new = fmaxf(m, top);
    const float keep = m_new == -INFINITY ? 1.f : expf(m - m_new);
    const float w = base ? expf(score - m_new) : 0.f;
    w_s[tid] = w;
    __syncthreads();
    m = m_new;
    l *= keep;
    acc *= keep;
    for (int i = 0; i < kSimpleThreads; ++i) {
      l += w_s[i];
      if (base_s[i] && tid < D) acc = fmaf(w_s[i], kv_value<D, Q4>(c, base_s[i] + c.half_bytes, row_s[i], tid), acc);
    }
  }
  if (tid < D) {
    const float o = l > 0.f ? acc / l : (l == 0.f ? 0.f : l);
    T* out = static_cast<T*>(p.o) + r * p.o_stride + (int64_t)h * D;
    if constexpr (sizeof(T) == 4) out[tid] = o;
    else out[tid] = f32_to_bf16_bits(o);
  }
}

template <int D, bool Q4, class T>
cudaError_t launch_simple(const KvAttnParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.nq, p.n);
  cfg.blockDim = dim3(kSimpleThreads);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kv_attn_simple<D, Q4, T>, p);
}

int check_attention(const dec_kv_cache* c, int n, int n_q_heads) {
  if (n < 0 || n > 65535) return fail_no_handle(DEC_ERR_ARG, "%d queries (0..65535)", n);
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || n_q_heads > 65536)
    return fail_no_handle(DEC_ERR_SHAPE, "%d query heads: a multiple of the %d KV heads", n_q_heads, c->n_kv_heads);
  return DEC_OK;
}

// Whether rows of `width` bytes at a + i * sa and at b + i * sb (i < n) share a byte.
bool rows_overlap(uintptr_t a, int64_t sa, uintptr_t b, int64_t sb, int64_t width, int n) {
  if (a + (n - 1) * sa + width <= b || b + (n - 1) * sb + width <= a) return false;
  if (sa != sb) return true;
  const int64_t d = (int64_t)(a > b ? a - b : b - a) % sa;
  return d < width || d > sa - width;
}

}  // namespace

extern "C" int dec_kv_attention_workspace(const dec_kv_cache* c, int n, int n_q_heads, size_t* bytes) {
  if (int rc = kv_check(c, false)) return rc;
  if (int rc = check_attention(c, n, n_q_heads)) return rc;
  if (!bytes) return fail_no_handle(DEC_ERR_ARG, "bytes is NULL");
  *bytes = 16;
  return DEC_OK;
}

extern "C" int dec_kv_attention(const dec_kv_cache* c, int layer, const void* q, void* o, int type, int64_t q_stride,
                                int64_t o_stride, const int32_t* seqs, int n, int n_q_heads, int window, int sinks,
                                float scale, void* workspace, size_t workspace_bytes, dec_stream_t stream) {
  if (int rc = kv_check(c, true)) return rc;
  if (int rc = check_attention(c, n, n_q_heads)) return rc;
  if (layer < 0 || layer >= c->n_layers) return fail_no_handle(DEC_ERR_ARG, "layer %d out of range", layer);
  if (type != DEC_IO_F32 && type != DEC_IO_BF16) return fail_no_handle(DEC_ERR_ARG, "unknown type %d", type);
  if (window < 0 || sinks < 0) return fail_no_handle(DEC_ERR_ARG, "window %d, sinks %d", window, sinks);
  if (!std::isfinite(scale)) return fail_no_handle(DEC_ERR_ARG, "the scale is not finite");
  if (!seqs && n > c->n_seqs) return fail_no_handle(DEC_ERR_ARG, "%d queries of %d sequences", n, c->n_seqs);
  if (n == 0) return DEC_OK;
  if (!q || !o) return fail_no_handle(DEC_ERR_ARG, "q or o is NULL");
  const int64_t size = type == DEC_IO_F32 ? 4 : 2, width = (int64_t)n_q_heads * c->head_dim;
  if (q_stride < width || o_stride < width || q_stride > (int64_t)1 << 40 || o_stride > (int64_t)1 << 40)
    return fail_no_handle(DEC_ERR_ARG, "q_stride or o_stride below the row's %lld elements", (long long)width);
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15) || (q_stride * size) % 16 ||
      (o_stride * size) % 16)
    return fail_no_handle(DEC_ERR_ARG, "q, o and their rows must be 16-byte aligned");
  if (rows_overlap(reinterpret_cast<uintptr_t>(q), q_stride * size, reinterpret_cast<uintptr_t>(o), o_stride * size,
                   width * size, n))
    return fail_no_handle(DEC_ERR_ARG, "o overlaps q");
  size_t need = 0;
  if (int rc = dec_kv_attention_workspace(c, n, n_q_heads, &need)) return rc;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) || workspace_bytes < need)
    return fail_no_handle(DEC_ERR_ARG, "the workspace must be 16-byte aligned and of %zu bytes", need);

  KvAttnParams p;
  p.c = kv_view(*c, layer);
  p.q = q;
  p.o = o;
  p.q_stride = q_stride;
  p.o_stride = o_stride;
  p.seqs = seqs;
  p.n = n;
  p.nq = n_q_heads;
  p.window = window;
  p.sinks = sinks;
  p.scale = scale != 0.f ? scale : (float)(1.0 / std::sqrt((double)c->head_dim));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool q4 = c->format == DEC_KV_Q4B32, f32 = type == DEC_IO_F32;
#define TLD_ATTN(D, Q) e = f32 ? launch_simple<D, Q, float>(p, s) : launch_simple<D, Q, uint16_t>(p, s)
  if (c->head_dim == 128) {
    if (q4) TLD_ATTN(128, true);
    else TLD_ATTN(128, false);
  } else {
    if (q4) TLD_ATTN(64, true);
    else TLD_ATTN(64, false);
  }
#undef TLD_ATTN
  if (e != cudaSuccess) return fail_no_handle(DEC_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
  return DEC_OK;
}
