// dec_kv_append and dec_kv_read: rows of a paged key/value cache from and to
// plain tensors, bf16 or in 4-bit blocks.  Also the checks shared by the
// dec_kv_ calls.
#include <cstdio>

#include "common.cuh"
#include "kv.h"

using namespace tld;

namespace tld {

int kv_check(const dec_kv_cache* c, bool memory) {
  if (!c) return fail_no_handle(DEC_ERR_ARG, "the cache is NULL");
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail_no_handle(DEC_ERR_SHAPE, "head_dim %d unsupported (64 or 128)", c->head_dim);
  if (c->page_rows < 16 || c->page_rows > 1024 || c->page_rows % 16)
    return fail_no_handle(DEC_ERR_SHAPE, "page_rows %d: a multiple of 16, 16..1024", c->page_rows);
  if (c->n_layers < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return fail_no_handle(DEC_ERR_SHAPE, "%d layers, %d KV heads", c->n_layers, c->n_kv_heads);
  if (c->n_pages < 1 || c->n_pages > (1 << 20) || c->n_seqs < 1 || c->n_seqs > 65536)
    return fail_no_handle(DEC_ERR_SHAPE, "%d pages, %d sequences (at most 2^20 and 65536)", c->n_pages, c->n_seqs);
  if (c->max_pages < 1 || (int64_t)c->max_pages * c->page_rows > (1 << 30))
    return fail_no_handle(DEC_ERR_SHAPE, "max_pages %d of %d rows (at most 2^30 rows)", c->max_pages, c->page_rows);
  if (c->format != DEC_KV_BF16 && c->format != DEC_KV_Q4B32)
    return fail_no_handle(DEC_ERR_ARG, "unknown cache format %d", c->format);
  if (memory) {
    if (!c->pool || !c->table || !c->lens || !c->refs || !c->status || !c->scratch)
      return fail_no_handle(DEC_ERR_ARG, "a pointer of the cache is NULL");
    const uintptr_t ints = reinterpret_cast<uintptr_t>(c->table) | reinterpret_cast<uintptr_t>(c->lens) |
                           reinterpret_cast<uintptr_t>(c->refs) | reinterpret_cast<uintptr_t>(c->status) |
                           reinterpret_cast<uintptr_t>(c->scratch);
    if ((reinterpret_cast<uintptr_t>(c->pool) & 15) || (ints & 3))
      return fail_no_handle(DEC_ERR_ARG, "the pool must be 16-byte aligned, the tables 4-byte aligned");
  }
  return DEC_OK;
}

KvView kv_view(const dec_kv_cache& c, int layer) {
  KvView v;
  v.head_bytes = (int64_t)c.page_rows * kv_row_bytes(c.head_dim, c.format == DEC_KV_Q4B32);
  v.half_bytes = v.head_bytes * c.n_kv_heads;
  v.page_bytes = 2 * v.half_bytes;
  v.pool = static_cast<uint8_t*>(c.pool) + (int64_t)layer * c.n_pages * v.page_bytes;
  v.table = c.table;
  v.lens = c.lens;
  v.refs = c.refs;
  v.status = c.status;
  v.scratch = c.scratch;
  v.n_pages = c.n_pages;
  v.n_seqs = c.n_seqs;
  v.max_pages = c.max_pages;
  v.page_rows = c.page_rows;
  v.nkv = c.n_kv_heads;
  return v;
}

}  // namespace tld

namespace {

constexpr int kRowWarps = 8;  // warps of a CTA of the row kernels

// Four fp32 values from / to the caller's type.
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&x)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&x)[4]) {
  uint2 w;
  w.x = f32_to_bf16_bits(x[0]) | (uint32_t)f32_to_bf16_bits(x[1]) << 16;
  w.y = f32_to_bf16_bits(x[2]) | (uint32_t)f32_to_bf16_bits(x[3]) << 16;
  *reinterpret_cast<uint2*>(p) = w;
}

// The code of x for a scale s > 0: the integer nearest to x / s, ties to even.
// The fp32 quotient can only err where it lands on a half: there the sign of
// x - (q +- 0.5) s, which one FMA gives exactly, decides.
__device__ __forceinline__ int q4_code(float x, float s) {
  float q = rintf(__fdiv_rn(x, s));
  if (fmaf(-(q + 0.5f), s, x) > 0.f) q += 1.f;
  else if (fmaf(-(q - 0.5f), s, x) < 0.f) q -= 1.f;
  return (int)fminf(fmaxf(q, -8.f), 7.f);
}

// The page row a token goes to, or null (with the status bit set where that is an error).
__device__ __forceinline__ uint8_t* kv_token_row(const KvView& c, const int32_t* seqs,
                                                 const int32_t* positions, int t, int which, int head,
                                                 int* row) {
  const int s = seqs ? seqs[t] : t;
  if (s < 0) return nullptr;
  int page = -1;
  if (s < c.n_seqs) {
    const int pos = positions ? positions[t] : c.lens[s] - 1;
    if (pos >= 0 && pos < c.max_pages * c.page_rows) {
      page = c.table[(int64_t)s * c.max_pages + pos / c.page_rows];
      *row = pos % c.page_rows;
    }
  }
  if (page < 0 || page >= c.n_pages) {
    atomicOr(c.status, DEC_KV_BAD_INDEX);
    return nullptr;
  }
  return c.pool + page * c.page_bytes + which * c.half_bytes + head * c.head_bytes;
}

// One row of K or V of one head takes D / 4 lanes, four dimensions 4 l .. 4 l + 3
// each: lane l = 8 b + g of a row holds the four dimensions of block b that
// share a 16-bit word of the row's codes, so the loads, the block maximum (8
// lanes) and the stores are all whole.
template <int D, bool Q4, class T, bool READ>
__global__ void __launch_bounds__(kRowWarps * 32) kv_rows(KvView c, T* k, T* v, int64_t stride,
                                                          const int32_t* seqs, const int32_t* positions,
                                                          int n) {
  constexpr int LANES = D / 4, NB = D / 32;
  const int l = threadIdx.x % LANES, b = l / 8, g = l % 8;
  const int64_t item = ((int64_t)blockIdx.x * kRowWarps * 32 + threadIdx.x) / LANES;
  const int per = 2 * c.nkv;
  const int64_t t = item / per;
  const bool in = t < n;
  const int which = (int)(item % per) / c.nkv, head = (int)(item % per) % c.nkv;
  int row = 0;
  uint8_t* base = in ? kv_token_row(c, seqs, positions, (int)t, which, head, &row) : nullptr;
  T* x_ptr = (which ? v : k) + t * stride + (int64_t)head * D + 4 * l;
  if constexpr (!Q4) {
    if (!base) return;
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + (int64_t)row * D + 4 * l;
    float x[4];
    if constexpr (READ) {
      load4(p, x);
      store4(x_ptr, x);
    } else {
      load4(x_ptr, x);
      store4(p, x);
    }
  } else {
    uint16_t* code_ptr = reinterpret_cast<uint16_t*>(base + (int64_t)row * (D / 2)) + g * NB + b;
    __half* scale_ptr = reinterpret_cast<__half*>(base + (int64_t)c.page_rows * (D / 2)) + (int64_t)row * NB + b;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (READ) {
      if (!base) return;
      const uint32_t w = *code_ptr;
      const float s = __half2float(*scale_ptr);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (float)((int)((w >> (4 * i)) & 15) - 8) * s;
      store4(x_ptr, x);
    } else {
      if (base) load4(x_ptr, x);
      uint32_t top = 0;  // largest magnitude of the block, as bits: order of the values, NaN and infinity last
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (!base) return;
      const bool finite = top < 0x7f800000u;
      const __half s = finite ? __float2half_rn(fminf(__fdiv_rn(__uint_as_float(top), 7.f), 65504.f))
                              : __ushort_as_half(0x7fff);
      const float sf = __half2float(s);
      uint32_t w = 0x8888u;
      if (finite && sf > 0.f) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= (uint32_t)(q4_code(x[i], sf) + 8) << (4 * i);
      }
      *code_ptr = (uint16_t)w;
      if (g == 0) *scale_ptr = s;
    }
  }
}

template <int D, bool Q4, class T, bool READ>
cudaError_t launch_rows(const KvView& c, void* k, void* v, int64_t stride, const int32_t* seqs,
                        const int32_t* positions, int n, cudaStream_t s) {
  const int64_t threads = (int64_t)n * 2 * c.nkv * (D / 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((threads + kRowWarps * 32 - 1) / (kRowWarps * 32)));
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kv_rows<D, Q4, T, READ>, c, static_cast<T*>(k), static_cast<T*>(v), stride, seqs,
                            positions, n);
}

template <bool READ>
int rows_call(const dec_kv_cache* c, int layer, void* k, void* v, int type, int64_t row_stride,
              const int32_t* seqs, const int32_t* positions, int n, dec_stream_t stream) {
  if (int rc = kv_check(c, true)) return rc;
  if (layer < 0 || layer >= c->n_layers) return fail_no_handle(DEC_ERR_ARG, "layer %d out of range", layer);
  if (type != DEC_IO_F32 && type != DEC_IO_BF16) return fail_no_handle(DEC_ERR_ARG, "unknown type %d", type);
  if (n < 0 || (!seqs && n > c->n_seqs))
    return fail_no_handle(DEC_ERR_ARG, "%d rows (without a list, one per sequence at most)", n);
  if (n == 0) return DEC_OK;
  if (!k || !v) return fail_no_handle(DEC_ERR_ARG, "k or v is NULL");
  const int64_t size = type == DEC_IO_F32 ? 4 : 2, width = (int64_t)c->n_kv_heads * c->head_dim;
  if (row_stride < width || row_stride > (int64_t)1 << 40)
    return fail_no_handle(DEC_ERR_ARG, "row_stride %lld below the row's %lld elements", (long long)row_stride,
                          (long long)width);
  if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) || (row_stride * size) % 16)
    return fail_no_handle(DEC_ERR_ARG, "k, v and their rows must be 16-byte aligned");
  if ((int64_t)n * 2 * width > (int64_t)1 << 38)
    return fail_no_handle(DEC_ERR_SHAPE, "%d rows are more than one launch takes", n);
  const KvView view = kv_view(*c, layer);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool q4 = c->format == DEC_KV_Q4B32, f32 = type == DEC_IO_F32;
#define TLD_ROWS(D, Q)                                                                                  \
  e = f32 ? launch_rows<D, Q, float, READ>(view, k, v, row_stride, seqs, positions, n, s)               \
          : launch_rows<D, Q, uint16_t, READ>(view, k, v, row_stride, seqs, positions, n, s)
  if (c->head_dim == 128) {
    if (q4) TLD_ROWS(128, true);
    else TLD_ROWS(128, false);
  } else {
    if (q4) TLD_ROWS(64, true);
    else TLD_ROWS(64, false);
  }
#undef TLD_ROWS
  if (e != cudaSuccess) return fail_no_handle(DEC_ERR_CUDA, "row kernel launch: %s", cudaGetErrorString(e));
  return DEC_OK;
}

}  // namespace

extern "C" int dec_kv_sizes(const dec_kv_cache* c, size_t* page_bytes, size_t* scratch_ints) {
  if (int rc = kv_check(c, false)) return rc;
  if (page_bytes) *page_bytes = (size_t)kv_view(*c, 0).page_bytes;
  if (scratch_ints) *scratch_ints = (size_t)kv_scratch_ints(c->n_pages, c->n_seqs);
  return DEC_OK;
}

extern "C" int dec_kv_append(const dec_kv_cache* c, int layer, const void* k, const void* v, int type,
                             int64_t row_stride, const int32_t* seqs, const int32_t* positions, int n,
                             dec_stream_t stream) {
  return rows_call<false>(c, layer, const_cast<void*>(k), const_cast<void*>(v), type, row_stride, seqs, positions, n,
                          stream);
}

extern "C" int dec_kv_read(const dec_kv_cache* c, int layer, void* k, void* v, int type, int64_t row_stride,
                           const int32_t* seqs, const int32_t* positions, int n, dec_stream_t stream) {
  return rows_call<true>(c, layer, k, v, type, row_stride, seqs, positions, n, stream);
}

extern "C" int dec_kv_status(const dec_kv_cache* c, int* bits, dec_stream_t stream) {
  if (bits) *bits = 0;
  if (int rc = kv_check(c, true)) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int flag = 0;
  cudaError_t e = cudaMemcpyAsync(&flag, c->status, sizeof flag, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && flag) {
    e = cudaMemsetAsync(c->status, 0, sizeof flag, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return fail_no_handle(DEC_ERR_CUDA, "reading the cache's status: %s", cudaGetErrorString(e));
  if (bits) *bits = flag;
  if (flag)
    return fail_no_handle(DEC_ERR_DEVICE, "the cache's kernels refused something (bits 0x%x:%s%s%s)", flag,
                          flag & DEC_KV_BAD_INDEX ? " index out of range" : "",
                          flag & DEC_KV_NO_PAGES ? " no free pages" : "",
                          flag & DEC_KV_BAD_LIST ? " bad list" : "");
  return DEC_OK;
}
