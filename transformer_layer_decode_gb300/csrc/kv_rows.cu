// dec_kv_append and dec_kv_read: rows of a paged key/value cache from and to
// plain tensors, bf16 or in 4-bit blocks.  Also the checks shared by the
// dec_kv_ calls.
#include <algorithm>
#include <cstdio>
#include <type_traits>

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
// Rounds of a warp, rows whose loads are under way together, where there are
// enough warps to fill the GPU; one otherwise.
constexpr int kRowRounds = 4;
constexpr int kFewRounds = 8192;  // (about a GPU full of warps)
// CTAs beyond which they take more tokens each (half or 1.5 times as many: up to
// 6 % slower).
constexpr int kManyCtas = 2400;

// The largest of three magnitudes; NaN if one is.
__device__ __forceinline__ float largest(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// The larger magnitudes of two bf16 pairs (with some sign); NaN if either is.
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// Two fp32 numbers handled by one instruction.
struct Two {
  uint64_t w;
  __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit Two(float a) : Two(a, a) {}
  __device__ __forceinline__ float2 get() const {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(w));
    return y;
  }
};
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.w) : "l"(b.w), "l"(c.w));
  return a;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.w) : "l"(b.w));
  return a;
}

// Eight values of the caller's type as they are loaded, their fp32 values, and
// the largest magnitude among them and those of four neighbouring lanes (NaN if
// one of them is).
template <class T>
struct Eight;
template <>
struct Eight<float> {
  float4 u, w;
  __device__ __forceinline__ void load(const float* p) {
    u = reinterpret_cast<const float4*>(p)[0], w = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
  }
  __device__ __forceinline__ float top() const {
    float y = largest(largest(largest(u.x, u.y, u.z), u.w, w.x), w.y, w.z);
    y = largest(y, w.w, __shfl_xor_sync(0xffffffffu, largest(y, w.w, 0.f), 1));
    return largest(y, __shfl_xor_sync(0xffffffffu, y, 2), 0.f);
  }
};
template <>
struct Eight<uint16_t> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = bf16lo(u.x), x[1] = bf16hi(u.x), x[2] = bf16lo(u.y), x[3] = bf16hi(u.y);
    x[4] = bf16lo(u.z), x[5] = bf16hi(u.z), x[6] = bf16lo(u.w), x[7] = bf16hi(u.w);
  }
  __device__ __forceinline__ float top() const {
    uint32_t y = larger2(larger2(u.x, u.y), larger2(u.z, u.w));
    y = larger2(y, __shfl_xor_sync(0xffffffffu, y, 1));
    y = larger2(y, __shfl_xor_sync(0xffffffffu, y, 2));
    return largest(bf16lo(y), bf16hi(y), 0.f);
  }
};
// wide: p is a multiple of 32 bytes, which one store then writes whole; two
// stores of half a sector each take longer (8185 rows of 32 heads of 128 read
// from 4-bit pages: 81 us, against 51).
__device__ __forceinline__ void store8(float* p, const float (&x)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}
__device__ __forceinline__ uint32_t pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8], bool) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7]));
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer

// 1 / s to a few 2^-24 of itself.
__device__ __forceinline__ float reciprocal(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  return y;
}

// Codes plus 8 of eight values for a scale s > 0, four bits each, lowest first:
// the integers nearest to x / s, ties to even, within [-8, 7].  The quotient takes
// one correction (Markstein's division): with a reciprocal that is off by 2^-23 of
// itself, r = r0 + (x - r0 s) / s is off from x / s by half a step of r and a
// millionth of a step.  x has 24 bits and s 11, so x / s is a half exactly, and then
// so is r, or it is away from every half by half a step and 2^-11 of that or more,
// and r is on the same side.  Scales below fp16's normal numbers, or at its top, can
// be too small for their block: there x is clamped.  Adding kMagic leaves
// the integer in a float's low bits, whose other bits leave the word as it is put
// together from its digits.  x[i] and x[4 + i], which are the same digit, go through
// each step in one instruction.
__device__ __forceinline__ uint32_t q4_codes(float (&x)[8], float s) {
  if (s < 6.103515625e-5f || s >= 65504.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -8.f * s), 7.f * s);
  }
  const Two inv(reciprocal(s)), minus(-s), magic(kMagic), zero(-0.f);
  uint32_t y0 = 0, y1 = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const Two u(x[i], x[4 + i]), r0 = fma2(u, inv, zero), r = fma2(fma2(r0, minus, u), inv, r0);
    const float2 m = add2(r, i ? magic : Two(kMagic + 34952.f)).get();  // 8 in every digit
    y0 = y0 * 16 + __float_as_uint(m.x), y1 = y1 * 16 + __float_as_uint(m.y);
  }
  return __byte_perm(y0, y1, 0x5410);
}

// x / 7, correctly rounded: the product with the rounded reciprocal and one FMA
// correction (Markstein's division; the quotient's remainder is exact).
__device__ __forceinline__ float seventh(float x) {
  constexpr float y = 1.f / 7;
  const float q = x * y;
  return fmaf(fmaf(-7.f, q, x), y, q);
}

constexpr int kMaxTokens = 32;  // of a CTA

// A CTA takes `tokens` tokens, looks up where each goes (a thread per token),
// and its warps take them in turn, ROUNDS rounds of 256 / D rows of a token
// (K's heads, then V's) at a time, so that these rows' loads are under way
// together.  A row takes D / 8 lanes, eight dimensions 8 l .. 8 l + 7 each:
// lane l = 4 b + j has the dimensions of block b that make up groups g = 2 j and
// 2 j + 1, two whole 16-bit words of the row's codes.
//
// What bounds it: 8185 rows of 32 heads of 128 in bf16, 172 MB with their 4-bit
// rows, are written in 37 us and read in 33, where the bytes take 26: latency (a
// CTA's look-up and the barrier behind it, then its rows' loads, then amax, scale,
// quotients and digits; issue is active in 67 and 59 %, the integer pipe in 53 and
// 57).  In fp32, 306 MB, 51 and 51 us (46); from and to bf16 pages, 268 MB, 43 (40),
// fp32 and bf16 pages, 402 MB, 61 and 62 (60).  Four rounds:
// two are 10 % slower, eight 15 % in fp32.
template <int D, bool Q4, class T, bool READ, int ROUNDS>
__global__ void __launch_bounds__(kRowWarps * 32) kv_rows(KvView c, T* k, T* v, int64_t stride,
                                                          const int32_t* seqs, const int32_t* positions,
                                                          int n, int tokens, int items_per_token, bool wide) {
  constexpr int LANES = D / 8, NB = D / 32, RPR = 32 / LANES;  // rows of a round
  __shared__ uint8_t* token_page[kMaxTokens];
  __shared__ int token_row[kMaxTokens];
  const int lane = threadIdx.x & 31, l = lane % LANES, b = l / 4, j = l % 4;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  if (threadIdx.x < tokens) {
    const int64_t t = t0 + threadIdx.x;
    uint8_t* at = nullptr;
    const int s = t < n ? (seqs ? seqs[t] : (int)t) : -1;
    if (s >= 0) {
      int page = -1;
      if (s < c.n_seqs) {
        const int pos = positions ? positions[t] : c.lens[s] - 1;
        if (pos >= 0 && pos < c.max_pages * c.page_rows) {
          page = c.table[(int64_t)s * c.max_pages + pos / c.page_rows];
          token_row[threadIdx.x] = pos % c.page_rows;
        }
      }
      if (page >= 0 && page < c.n_pages) at = c.pool + page * c.page_bytes;
      else atomicOr(c.status, DEC_KV_BAD_INDEX);
    }
    token_page[threadIdx.x] = at;
  }
  __syncthreads();
  const int last = 2 * c.nkv - 1;
  int token = (threadIdx.x >> 5) / items_per_token, part = (threadIdx.x >> 5) % items_per_token;
  for (; token < tokens; part += kRowWarps) {
    if (part >= items_per_token) {
      token += part / items_per_token, part %= items_per_token;
      if (token >= tokens) break;
    }
    uint8_t* base = token_page[token];
    if (!base) continue;
    const int row = token_row[token], page_rows = c.page_rows, nkv = c.nkv;
    if (!KV_IN_BOUNDS(c, token < kMaxTokens && t0 + token < n && part >= 0 && row >= 0 && row < page_rows &&
                             base >= c.pool && base + c.page_bytes <= c.pool + c.n_pages * c.page_bytes &&
                             2 * nkv * c.head_bytes == c.page_bytes))
      continue;
    const uint32_t head_bytes = (uint32_t)c.head_bytes;
    const int first = part * (ROUNDS * RPR) + lane / LANES;
    // (lanes past the last row take it once more: the same bytes to the same place)
    auto round = [&](int i) { return min(first + i * RPR, last); };
    T* k_at = k + (t0 + token) * stride + 8 * l;
    T* v_at = v + (t0 + token) * stride + 8 * l - nkv * D;
    auto mine = [&](int at) { return (at < nkv ? k_at : v_at) + at * D; };  // the caller's
    // in the page: bf16 values, or two words of codes, 2 NB bytes apart, and a scale
    auto head = [&](int at) { return (uint64_t)(uint32_t)at * head_bytes; };
    uint8_t* values = base + row * kv_row_bytes(D, false) + 16 * l;
    uint8_t* words = base + row * (D / 2) + 4 * j * NB + 2 * b;
    uint8_t* scales = base + page_rows * (D / 2) + (row * NB + b) * 2;
    if constexpr (!READ || !Q4) {
      Eight<std::conditional_t<READ, uint16_t, T>> in[ROUNDS];
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const int at = round(i);
        if constexpr (READ) in[i].load(reinterpret_cast<const uint16_t*>(values + head(at)));
        else in[i].load(mine(at));
      }
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const int at = round(i);
        float x[8];
        in[i].values(x);
        if constexpr (READ) {
          store8(mine(at), x, wide);
        } else if constexpr (!Q4) {
          store8(reinterpret_cast<uint16_t*>(values + head(at)), x, false);
        } else {
          const float top = in[i].top();  // the block's largest magnitude
          const bool finite = top < INFINITY;
          const __half s16 = finite ? __float2half_rn(fminf(seventh(top), 65504.f)) : __ushort_as_half(0x7fff);
          const float f = __half2float(s16);
          // (where f is 0 every |x| is far below 1/2)
          const uint32_t codes = q4_codes(x, f > 0.f ? f : 1.f), w = finite ? codes : 0x88888888u;
          uint16_t* to = reinterpret_cast<uint16_t*>(words + head(at));
          to[0] = (uint16_t)w;
          to[NB] = (uint16_t)(w >> 16);
          if (j == 0) *reinterpret_cast<__half*>(scales + head(at)) = s16;
        }
      }
    } else {
      uint32_t codes[ROUNDS];
      __half scale[ROUNDS];
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const int at = round(i);
        const uint16_t* w = reinterpret_cast<const uint16_t*>(words + head(at));
        codes[i] = w[0] | (uint32_t)w[NB] << 16;
        scale[i] = *reinterpret_cast<const __half*>(scales + head(at));
      }
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const float f = __half2float(scale[i]);
        float x[8];
#pragma unroll
        for (int m = 0; m < 8; ++m)  // 2^23 + n, less 2^23 + 8
          x[m] = (__int_as_float(0x4b000000 | (codes[i] >> (4 * m) & 15)) - 8388616.f) * f;
        store8(mine(round(i)), x, wide);
      }
    }
  }
}

// Reads and clears the status in one step: bits that calls on other streams set in
// the meantime are in this answer or in the next.
__global__ void kv_take_status(int32_t* status, int32_t* taken) { *taken = atomicExch(status, 0); }

template <int D, bool Q4, class T, bool READ>
cudaError_t launch_rows(const KvView& c, void* k, void* v, int64_t stride, const int32_t* seqs,
                        const int32_t* positions, int n, cudaStream_t s) {
  constexpr int kPerRound = 256 / D;
  const bool few = (int64_t)n * 2 * c.nkv / kPerRound < kFewRounds;
  const int per_item = kPerRound * (few ? 1 : kRowRounds);
  const int items = (2 * c.nkv + per_item - 1) / per_item;
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | stride * sizeof(T)) & 31) == 0;
  // enough tokens for every warp of a CTA, or a multiple where there are CTAs enough
  const int least = (kRowWarps + items - 1) / items;
  const int tokens = std::min(std::max((n / kManyCtas + least - 1) / least, 1) * least, kMaxTokens);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n + tokens - 1) / tokens));
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, few ? kv_rows<D, Q4, T, READ, 1> : kv_rows<D, Q4, T, READ, kRowRounds>, c,
                            static_cast<T*>(k), static_cast<T*>(v), stride, seqs, positions, n, tokens, items, wide);
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
  if (READ && kv_rows_overlap(reinterpret_cast<uintptr_t>(k), row_stride * size, reinterpret_cast<uintptr_t>(v),
                              row_stride * size, width * size, n))
    return fail_no_handle(DEC_ERR_ARG, "k overlaps v");
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
  int word[2] = {0, 0};
  static_assert(kKvScratchStatus == kKvScratchLine + 1, "copied together");
  int32_t* taken = c->scratch + kKvScratchStatus;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = cfg.blockDim = dim3(1);
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_take_status, c->status, taken);
  if (e == cudaSuccess) e = cudaMemcpyAsync(word, taken - 1, sizeof word, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail_no_handle(DEC_ERR_CUDA, "reading the cache's status: %s", cudaGetErrorString(e));
  const int flag = word[1];
  if (bits) *bits = flag;
  if (flag & DEC_KV_BAD_BOUNDS)
    return fail_no_handle(DEC_ERR_DEVICE, "an index check of the cache's kernels failed at line %d (bits 0x%x)", word[0],
                          flag);
  if (flag)
    return fail_no_handle(DEC_ERR_DEVICE, "the cache's kernels refused something (bits 0x%x:%s%s%s)", flag,
                          flag & DEC_KV_BAD_INDEX ? " index out of range" : "",
                          flag & DEC_KV_NO_PAGES ? " no free pages" : "",
                          flag & DEC_KV_BAD_LIST ? " bad list" : "");
  return DEC_OK;
}
