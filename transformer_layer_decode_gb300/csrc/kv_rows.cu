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
constexpr int kRowRounds = 4; // rounds of a warp: rows whose loads are under way together

// Eight fp32 values from / to the caller's type.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 u = reinterpret_cast<const float4*>(p)[0], w = reinterpret_cast<const float4*>(p)[1];
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  x[0] = bf16lo(u.x), x[1] = bf16hi(u.x), x[2] = bf16lo(u.y), x[3] = bf16hi(u.y);
  x[4] = bf16lo(u.z), x[5] = bf16hi(u.z), x[6] = bf16lo(u.w), x[7] = bf16hi(u.w);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ uint32_t pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7]));
}

// Codes plus 8 of eight values for a scale s > 0, four bits each, lowest first:
// the integers nearest to x / s, ties to even, within [-8, 7].  r = x * (1 / s)
// is off by a few 2^-24 of itself, so its nearest integer q is the answer or,
// next to a half, a neighbour; the remainder e = x - q s is exact (it has no
// bits below x's and is below s), and |e| against s / 2 decides: past it, or on
// it with q odd, q moves one on.  EDGE: also for scales so small or so large
// that |x / s| passes 7.5 (s below fp16's normal numbers, or at its top).
template <bool EDGE>
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[8], float s) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  const float inv = 1.f / s;
  const int half = __float_as_int(0.5f * s);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float r = x[i] * inv;
    if (EDGE) r = fminf(fmaxf(r, -8.f), 7.f);
    const float m = r + kMagic, e = fmaf(-(m - kMagic), s, x[i]);
    int q = __float_as_int(m) - __float_as_int(kMagic);
    if (fabsf(e) > __int_as_float(half - (q & 1))) q += e > 0.f ? 1 : -1;
    if (EDGE) q = min(max(q, -8), 7);
    w |= (uint32_t)(q + 8) << (4 * i);
  }
  return w;
}

// A warp takes one token and kRowRounds rounds of 256 / D of its rows (K's
// heads, then V's), so that the token's page is looked up once and the rows'
// loads are under way together.  A row takes D / 8 lanes, eight dimensions
// 8 l .. 8 l + 7 each: lane l = 4 b + j has the dimensions of block b that make
// up groups g = 2 j and 2 j + 1, two whole 16-bit words of the row's codes.
//
// What bounds it: reading or writing the caller's rows, by bytes, and writing
// 4-bit rows the instructions besides (about 14 a value).
template <int D, bool Q4, class T, bool READ>
__global__ void __launch_bounds__(kRowWarps * 32) kv_rows(KvView c, T* k, T* v, int64_t stride,
                                                          const int32_t* seqs, const int32_t* positions,
                                                          int n, int warps_per_token) {
  constexpr int LANES = D / 8, NB = D / 32, RPR = 32 / LANES;  // rows of a round
  const int lane = threadIdx.x & 31, l = lane % LANES, b = l / 4, j = l % 4;
  const uint32_t warp = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const uint32_t t = warp / warps_per_token;
  if (t >= (uint32_t)n) return;
  const int s = seqs ? seqs[t] : (int)t;
  if (s < 0) return;
  int page = -1, row = 0;
  if (s < c.n_seqs) {
    const int pos = positions ? positions[t] : c.lens[s] - 1;
    if (pos >= 0 && pos < c.max_pages * c.page_rows) {
      page = c.table[(int64_t)s * c.max_pages + pos / c.page_rows];
      row = pos % c.page_rows;
    }
  }
  if (page < 0 || page >= c.n_pages) {
    if (lane == 0) atomicOr(c.status, DEC_KV_BAD_INDEX);
    return;
  }
  // (no lane of the warp has left)
  const int first = (warp % warps_per_token) * (kRowRounds * RPR) + lane / LANES;
  uint8_t* base = c.pool + page * c.page_bytes;
  const int64_t token = t * stride + 8 * l;
  float x[kRowRounds][8];
  if constexpr (!READ || !Q4) {
#pragma unroll
    for (int i = 0; i < kRowRounds; ++i) {
      const int at = first + i * RPR, head = at < c.nkv ? at : at - c.nkv;
      if (at >= 2 * c.nkv) continue;
      T* mine = (at < c.nkv ? k : v) + token + (int64_t)head * D;
      uint16_t* bf = reinterpret_cast<uint16_t*>(base + at * c.head_bytes) + row * D + 8 * l;
      if constexpr (READ) load8(bf, x[i]);
      else load8(mine, x[i]);
    }
  }
  if constexpr (!Q4) {
#pragma unroll
    for (int i = 0; i < kRowRounds; ++i) {
      const int at = first + i * RPR, head = at < c.nkv ? at : at - c.nkv;
      if (at >= 2 * c.nkv) continue;
      T* mine = (at < c.nkv ? k : v) + token + (int64_t)head * D;
      uint16_t* bf = reinterpret_cast<uint16_t*>(base + at * c.head_bytes) + row * D + 8 * l;
      if constexpr (READ) store8(mine, x[i]);
      else store8(bf, x[i]);
    }
  } else if constexpr (READ) {
    uint32_t codes[kRowRounds];
    __half scale[kRowRounds];
#pragma unroll
    for (int i = 0; i < kRowRounds; ++i) {
      const int at = first + i * RPR;
      if (at >= 2 * c.nkv) continue;
      const uint8_t* head = base + at * c.head_bytes;
      const uint16_t* words = reinterpret_cast<const uint16_t*>(head + row * (D / 2)) + 2 * j * NB + b;
      codes[i] = words[0] | (uint32_t)words[NB] << 16;
      scale[i] = reinterpret_cast<const __half*>(head + (int64_t)c.page_rows * (D / 2))[row * NB + b];
    }
#pragma unroll
    for (int i = 0; i < kRowRounds; ++i) {
      const int at = first + i * RPR, head = at < c.nkv ? at : at - c.nkv;
      if (at >= 2 * c.nkv) continue;
      const float f = __half2float(scale[i]);
#pragma unroll
      for (int m = 0; m < 8; ++m)  // 2^23 + n, less 2^23 + 8
        x[i][m] = (__int_as_float(0x4b000000 | (codes[i] >> (4 * m) & 15)) - 8388616.f) * f;
      store8((at < c.nkv ? k : v) + token + (int64_t)head * D, x[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRowRounds; ++i) {
      const int at = first + i * RPR;
      const bool on = at < 2 * c.nkv;
      uint32_t top = 0;  // the block's largest magnitude, as bits: in the order of the values, infinity and NaN last
      if (on) {
#pragma unroll
        for (int m = 0; m < 8; ++m) top = max(top, __float_as_uint(x[i][m]) & 0x7fffffffu);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (!on) continue;
      const bool finite = top < 0x7f800000u;
      const __half s16 = finite ? __float2half_rn(fminf(__fdiv_rn(__uint_as_float(top), 7.f), 65504.f))
                                : __ushort_as_half(0x7fff);
      const float f = __half2float(s16);
      uint32_t w = 0x88888888u;
      if (f >= 6.103515625e-5f && f < 65504.f) w = q4_codes<false>(x[i], f);
      else if (f > 0.f) w = q4_codes<true>(x[i], f);  // (not where f is NaN)
      uint8_t* head = base + at * c.head_bytes;
      uint16_t* words = reinterpret_cast<uint16_t*>(head + row * (D / 2)) + 2 * j * NB + b;
      words[0] = (uint16_t)w;
      words[NB] = (uint16_t)(w >> 16);
      if (j == 0) reinterpret_cast<__half*>(head + (int64_t)c.page_rows * (D / 2))[row * NB + b] = s16;
    }
  }
}

template <int D, bool Q4, class T, bool READ>
cudaError_t launch_rows(const KvView& c, void* k, void* v, int64_t stride, const int32_t* seqs,
                        const int32_t* positions, int n, cudaStream_t s) {
  constexpr int kPerWarp = kRowRounds * (256 / D);
  const int warps_per_token = (2 * c.nkv + kPerWarp - 1) / kPerWarp;
  const int64_t warps = (int64_t)n * warps_per_token;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kRowWarps - 1) / kRowWarps));
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kv_rows<D, Q4, T, READ>, c, static_cast<T*>(k), static_cast<T*>(v), stride, seqs,
                            positions, n, warps_per_token);
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
  if ((int64_t)n * c->n_kv_heads > (int64_t)1 << 30)
    return fail_no_handle(DEC_ERR_SHAPE, "%d rows of %d heads (at most 2^30 in all)", n, c->n_kv_heads);
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
