// dec_kv_append and dec_kv_read: rows of a paged key/value cache from and to
// plain tensors, bf16 or in 4-bit blocks (and 8-bit rows read; kv_write8.cu writes
// them), and dec_kv_append_rotated.  Also the checks shared by the dec_kv_ calls.
#include <algorithm>
#include <cstdio>
#include <type_traits>

#include "common.cuh"
#include "kv.h"
#include "rope.cuh"
#include "rows.cuh"

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
  if (c->format != DEC_KV_BF16 && c->format != DEC_KV_Q4B32 && c->format != DEC_KV_Q8T16)
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
  v.head_bytes = (int64_t)c.page_rows * kv_row_bytes(c.head_dim, c.format);
  v.half_bytes = v.head_bytes * c.n_kv_heads;
  if (c.format == DEC_KV_Q8T16)
    v.half_bytes = (v.half_bytes + (int64_t)(c.page_rows / kBlockRows) * 4 * c.n_kv_heads + 63) / 64 * 64;
  v.page_bytes = 2 * v.half_bytes;
  v.pool = static_cast<uint8_t*>(c.pool) + (int64_t)layer * c.n_pages * v.page_bytes;
  v.table = c.table;
  v.lens = c.lens;
  v.refs = c.refs;
  v.status = c.status;
  v.scratch = c.scratch;
  v.owners = c.scratch ? c.scratch + kv_scratch_ints(c.n_pages, c.n_seqs) + (int64_t)layer * c.n_pages * c.page_rows : nullptr;
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
constexpr int kTurnedRounds = 2;  // of rows of which keys are rotated, whose partners are loaded too
constexpr int kFewRounds = 8192;  // (about a GPU full of warps)
// CTAs beyond which they take more tokens each (half or 1.5 times as many: up to
// 6 % slower).
constexpr int kManyCtas = 2400;
// Rotated rows: rounds of a CTA's warps at most.
constexpr int kTurnedTurns = 6;

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

// Eight values of a block of 32 whose largest magnitude is `top`: their codes to two words
// of the row, 2 NB bytes apart, and (leads) the block's scale.
template <int NB>
__device__ __forceinline__ void put_q4(float (&x)[8], float top, uint8_t* words, uint8_t* scale, bool leads) {
  const bool finite = top < INFINITY;
  const __half s16 = finite ? __float2half_rn(fminf(seventh(top), 65504.f)) : __ushort_as_half(0x7fff);
  const float f = __half2float(s16);
  // (where f is 0 every |x| is far below 1/2)
  const uint32_t codes = q4_codes(x, f > 0.f ? f : 1.f), w = finite ? codes : 0x88888888u;
  uint16_t* to = reinterpret_cast<uint16_t*>(words);
  to[0] = (uint16_t)w;
  to[NB] = (uint16_t)(w >> 16);
  if (leads) *reinterpret_cast<__half*>(scale) = s16;
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
// rows, are written in 38 us and read in 33, where the bytes take 26: latency (a
// CTA's look-up and the barrier behind it, then its rows' loads, then amax, scale,
// quotients and digits; issue is active in 67 and 59 %, the integer pipe in 53 and
// 57).  In fp32, 306 MB, 51 and 51 us (46); from and to bf16 pages, 268 MB, 43 (40),
// fp32 and bf16 pages, 402 MB, 61 and 62 (60).  Four rounds:
// two are 10 % slower, eight 15 % in fp32.  (The view as a grid constant: 48 registers and a
// fifth CTA an SM; a copy of it, 52, and rows written to 4-bit pages 41 us for 38.  8-bit
// pages are read from a copy: 34.4 us for 35.5.)
template <int D, int F, class T, bool READ, int ROUNDS>
__global__ void __launch_bounds__(kRowWarps * 32) kv_rows(const __grid_constant__ KvView view, T* k, T* v,
                                                          int64_t stride, const int32_t* seqs,
                                                          const int32_t* positions, int n, int tokens,
                                                          int items_per_token, bool wide) {
  std::conditional_t<F == KV_Q8, const KvView, const KvView&> c = view;
  constexpr int LANES = D / 8, NB = D / 32, RPR = 32 / LANES;  // rows of a round
  __shared__ uint8_t* token_page[kMaxTokens];
  __shared__ int token_row[kMaxTokens];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, l = lane % LANES, b = l / 4, j = l % 4;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  if (threadIdx.x < tokens) {
    const int64_t t = t0 + threadIdx.x;
    const KvPlace at = kv_place(c, seqs, positions, t, n);
    token_row[threadIdx.x] = at.row;
    token_page[threadIdx.x] = at.page;
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
                             (F == KV_Q8 || 2 * nkv * c.head_bytes == c.page_bytes)))
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
    uint8_t* values = base + row * kv_row_bytes(D, KV_BF16) + 16 * l;
    uint8_t* words = base + row * (D / 2) + 4 * j * NB + 2 * b;
    uint8_t* scales = base + page_rows * (D / 2) + (row * NB + b) * 2;
    if constexpr (READ && F == KV_Q8) {
      uint2 codes[ROUNDS];
      float scale[ROUNDS];
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const int at = round(i), h = at < nkv ? at : at - nkv;
        const uint8_t* half = base + (at < nkv ? 0 : c.half_bytes);
        codes[i] = *reinterpret_cast<const uint2*>(half + (uint64_t)(uint32_t)h * head_bytes + row * D + 8 * l);
        scale[i] = *reinterpret_cast<const float*>(half + (uint64_t)(uint32_t)nkv * head_bytes +
                                                   4 * ((int64_t)h * (page_rows / kBlockRows) + row / kBlockRows));
      }
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        float x[8];
#pragma unroll
        for (int m = 0; m < 8; ++m)  // 2^23 + byte, less 2^23 + 128
          x[m] = (__uint_as_float(__byte_perm(m < 4 ? codes[i].x : codes[i].y, 0x4b000000u, 0x7440 | (m & 3))) - 8388736.f) *
                 scale[i];
        store8(mine(round(i)), x, wide);
      }
    } else if constexpr (!READ || F == KV_BF16) {
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
        } else if constexpr (F == KV_BF16) {
          store8(reinterpret_cast<uint16_t*>(values + head(at)), x, false);
        } else {
          put_q4<NB>(x, in[i].top(), words + head(at), scales + head(at), j == 0);
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

// The rows of a step, as kv_rows writes them: the first `blocks` CTAs rotate and write keys
// and write values, the others rotate queries.  Many rows are loaded before it is known
// where they go and how they turn (8185 rows of 32 heads of fp32 to bf16 pages 79 -> 72 us),
// those of bf16 also the next ones before these are coded (4093 rows of 8 heads 15.0 -> 11.7;
// of fp32 that takes the registers of a third CTA an SM: 88).  CTAs: of an SM; of many rows of
// bf16 three, which leaves them the registers for that (8185 rows of 32 heads to bf16 pages
// 56 us, four 64), but four beside queries, whose CTAs have to fit as well (4093 rows of 8
// heads and 32 of queries 23 us, three 26); of fp32 four (8185 rows 68 us, three 72).
template <int D, int F, class T, int ROUNDS, int CTAS>
__global__ void __launch_bounds__(kRowWarps * 32, CTAS)
    kv_rows_rotated(const __grid_constant__ KvView c, const T* k, const T* v, int64_t stride, const int32_t* seqs,
                    const int32_t* positions, int n, int tokens, int items_per_token, int blocks,
                    const __grid_constant__ RopeRows q) {
  constexpr int LANES = D / 8, NB = D / 32, RPR = 32 / LANES;
  constexpr bool FIRST = ROUNDS > 1, AHEAD = FIRST && sizeof(T) == 2;
  extern __shared__ __align__(16) float q_angles[];
  __shared__ KvPlace place[kMaxTokens];
  __shared__ __align__(16) float angles[2][kMaxTokens * (D / 2)];  // cosines, sines
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= blocks) {
    rope_rows<T>(q, blockIdx.x - blocks, q_angles, [&](int64_t t) {
      const KvPlace at = kv_place(c, seqs, positions, t, n);
      return at.page ? at.pos : -1;
    });
    return;
  }
  const int lane = threadIdx.x & 31, l = lane % LANES, b = l / 4, j = l % 4, nkv = c.nkv, last = 2 * nkv - 1;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  struct Item {  // a warp's: ROUNDS rounds of rows of a token
    int token, part;
    Piece<T, true> in[ROUNDS];
  };
  // (lanes past the last row take it once more: the same bytes to the same place)
  auto round = [&](const Item& y, int i) { return min((y.part * ROUNDS + i) * RPR + lane / LANES, last); };
  auto row_of = [&](const Item& y, int at) {
    return (at < nkv ? k + at * D : v + (at - nkv) * D) + (t0 + y.token) * stride;
  };
  auto fetch = [&](int item) {
    Item y;
    y.token = item / items_per_token, y.part = item % items_per_token;
    if (y.token < tokens && t0 + y.token < n) {
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const int at = round(y, i);
        if (at < nkv) y.in[i].load(row_of(y, at), l, q.r);
        else y.in[i].own.load(row_of(y, at) + 8 * l);
      }
    }
    return y;
  };
  Item now;
  if (FIRST) now = fetch(threadIdx.x >> 5);
  if (threadIdx.x < tokens) place[threadIdx.x] = kv_place(c, seqs, positions, t0 + threadIdx.x, n);
  __syncthreads();
  const int half = q.r.rot / 2;
  for (int e = threadIdx.x; e < tokens * half; e += kRowWarps * 32) {
    const int t = e / half, i = e - t * half;
    if (!place[t].page) continue;
    const float2 y = rope_angle(q.r, place[t].pos, i);
    const int at = angle_at<D>(t, i);
    angles[0][at] = y.x, angles[1][at] = y.y;
  }
  __syncthreads();
  for (int item = threadIdx.x >> 5; item < tokens * items_per_token; item += kRowWarps) {
    Item next;
    if (AHEAD) next = fetch(item + kRowWarps);
    else if (!FIRST) now = fetch(item);
    const KvPlace at_token = place[now.token];
    if (at_token.page && KV_IN_BOUNDS(c, now.token < kMaxTokens && t0 + now.token < n && at_token.row >= 0 &&
                                             at_token.row < c.page_rows && at_token.page >= c.pool &&
                                             at_token.page + c.page_bytes <= c.pool + c.n_pages * c.page_bytes &&
                                             2 * nkv * c.head_bytes == c.page_bytes)) {
      const float* cs = angles[0] + now.token * (D / 2);
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const int at = round(now, i);
        uint8_t* head = at_token.page + (uint64_t)(uint32_t)at * (uint32_t)c.head_bytes;
        float x[8];
        if (at < nkv) turned<D>(now.in[i], x, row_of(now, at), l, q.r, cs, cs + kMaxTokens * (D / 2));
        else now.in[i].own.values(x);
        if constexpr (F == KV_BF16) {
          store8(reinterpret_cast<uint16_t*>(head + at_token.row * (2 * D) + 16 * l), x, false);
        } else {
          Eight<float> all;
          all.set(x);
          put_q4<NB>(x, all.top(), head + at_token.row * (D / 2) + 4 * j * NB + 2 * b,
                     head + c.page_rows * (D / 2) + (at_token.row * NB + b) * 2, j == 0);
        }
      }
    }
    if (AHEAD) now = next;
    else if (FIRST) now = fetch(item + kRowWarps);
  }
}

// Reads and clears the status in one step: bits that calls on other streams set in
// the meantime are in this answer or in the next.
__global__ void kv_take_status(int32_t* status, int32_t* taken) { *taken = atomicExch(status, 0); }

// Tokens of a CTA that rotates many rows, a multiple of `least`.  Its beginning, with the
// angles of its tokens, takes as long as two of its warps' turns, and the last CTAs to begin
// should have others beside them: so the least of waves times their length (8 heads of
// fp32, 4093 rows: 8 tokens 12.9 us, 12 15.6, 2 16.2; 2500 rows: 6 tokens 8.9, 12 11.3).  More
// than 6 turns seldom help (8185 rows of 32 heads of bf16: 3 tokens 55 us, 6 52, 12 57, 16 68).
inline int turned_tokens(int n, int least, int items, int resident) {
  int best = least;
  int64_t cost = INT64_MAX;
  for (int tokens = least; tokens <= kMaxTokens; tokens += least) {
    const int turns = (tokens * items + kRowWarps - 1) / kRowWarps;
    if (turns > kTurnedTurns && tokens > least) break;
    const int64_t ctas = (n + (int64_t)tokens - 1) / tokens, waves = (ctas + resident - 1) / resident;
    if (waves * (turns + 2) < cost) cost = waves * (turns + 2), best = tokens;
  }
  return best;
}

template <int D, int F, class T, bool READ>
cudaError_t launch_rows(const KvView& c, void* k, void* v, int64_t stride, const int32_t* seqs,
                        const int32_t* positions, int n, const RopeRows* q, cudaStream_t s) {
  constexpr int kPerRound = 256 / D;
  const bool few = (int64_t)n * 2 * c.nkv / kPerRound < kFewRounds;
  const int per_item = kPerRound * (few ? 1 : q ? kTurnedRounds : kRowRounds);
  const int items = (2 * c.nkv + per_item - 1) / per_item;
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | stride * sizeof(T)) & 31) == 0;
  // enough tokens for every warp of a CTA, or a multiple where there are CTAs enough
  const int least = (kRowWarps + items - 1) / items;
  int tokens = std::min(std::max((n / kManyCtas + least - 1) / least, 1) * least, kMaxTokens);
  const int turned_ctas = sizeof(T) == 2 && q && !q->n ? 3 : 4;
  if (q && !few) tokens = turned_tokens(n, least, items, turned_ctas * kSms);
  const int blocks = (n + tokens - 1) / tokens;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.stream = s;
  const BehindLast behind(&cfg);
  if constexpr (!READ) {
    if (q) {
      RopeRows rows = *q;
      if (rows.n) {
        cfg.gridDim.x += (unsigned)rope_cut(rows);
        cfg.dynamicSmemBytes = rope_smem(rows);
      }
      auto kernel = kv_rows_rotated<D, F, T, 1, 4>;
      if (!few) kernel = kv_rows_rotated<D, F, T, kTurnedRounds, 4>;
      if constexpr (sizeof(T) == 2)
        if (!few && turned_ctas == 3) kernel = kv_rows_rotated<D, F, T, kTurnedRounds, 3>;
      return cudaLaunchKernelEx(&cfg, kernel, c, static_cast<const T*>(k), static_cast<const T*>(v), stride, seqs,
                                positions, n, tokens, items, blocks, rows);
    }
  }
  return cudaLaunchKernelEx(&cfg, few ? kv_rows<D, F, T, READ, 1> : kv_rows<D, F, T, READ, kRowRounds>, c,
                            static_cast<T*>(k), static_cast<T*>(v), stride, seqs, positions, n, tokens, items, wide);
}

template <int D, class T, bool READ>
cudaError_t launch_format(int format, const KvView& c, void* k, void* v, int64_t stride, const int32_t* seqs,
                          const int32_t* positions, int n, const RopeRows* q, cudaStream_t s) {
  if (format == KV_Q4) return launch_rows<D, KV_Q4, T, READ>(c, k, v, stride, seqs, positions, n, q, s);
  if (format == KV_BF16) return launch_rows<D, KV_BF16, T, READ>(c, k, v, stride, seqs, positions, n, q, s);
  if constexpr (READ) return launch_rows<D, KV_Q8, T, true>(c, k, v, stride, seqs, positions, n, q, s);
  else return kv_write8(c, D, sizeof(T) == 4, k, v, stride, seqs, positions, n, q, s);
}

// q: the queries that an append rotates, and its rotation (of no queries: n = 0).
template <bool READ>
int rows_call(const dec_kv_cache* c, int layer, void* k, void* v, int type, int64_t row_stride,
              const int32_t* seqs, const int32_t* positions, int n, const RopeRows* q, dec_stream_t stream) {
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
  if (q && q->n) {
    const uintptr_t out = reinterpret_cast<uintptr_t>(q->out);
    for (const void* x : {k, v})
      if (kv_rows_overlap(out, q->out_stride * size, (int64_t)q->heads * q->d * size, reinterpret_cast<uintptr_t>(x),
                          row_stride * size, width * size, n))
        return fail_no_handle(DEC_ERR_ARG, "q_out overlaps k or v");
  }
  const KvView view = kv_view(*c, layer);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = type == DEC_IO_F32;
  cudaError_t e;
#define TLD_ROWS(D)                                                                                               \
  e = f32 ? launch_format<D, float, READ>(c->format, view, k, v, row_stride, seqs, positions, n, q, s)            \
          : launch_format<D, uint16_t, READ>(c->format, view, k, v, row_stride, seqs, positions, n, q, s)
  if (c->head_dim == 128) TLD_ROWS(128);
  else TLD_ROWS(64);
#undef TLD_ROWS
  if (e != cudaSuccess) return fail_no_handle(DEC_ERR_CUDA, "row kernel launch: %s", cudaGetErrorString(e));
  return DEC_OK;
}

// What every call on rows checks first.
int rows_check(const dec_kv_cache* c, int layer, int type, const int32_t* seqs, int n) {
  if (int rc = kv_check(c, true)) return rc;
  if (layer < 0 || layer >= c->n_layers) return fail_no_handle(DEC_ERR_ARG, "layer %d out of range", layer);
  if (type != DEC_IO_F32 && type != DEC_IO_BF16) return fail_no_handle(DEC_ERR_ARG, "unknown type %d", type);
  if (n < 0 || (!seqs && n > c->n_seqs))
    return fail_no_handle(DEC_ERR_ARG, "%d rows (without a list, one per sequence at most)", n);
  return DEC_OK;
}

}  // namespace

extern "C" int dec_kv_sizes(const dec_kv_cache* c, size_t* page_bytes, size_t* scratch_ints) {
  if (int rc = kv_check(c, false)) return rc;
  if (page_bytes) *page_bytes = (size_t)kv_view(*c, 0).page_bytes;
  if (scratch_ints) {
    *scratch_ints = (size_t)kv_scratch_ints(c->n_pages, c->n_seqs);
    if (c->format == DEC_KV_Q8T16) *scratch_ints += (size_t)c->n_layers * c->n_pages * c->page_rows;
  }
  return DEC_OK;
}

extern "C" int dec_kv_append(const dec_kv_cache* c, int layer, const void* k, const void* v, int type,
                             int64_t row_stride, const int32_t* seqs, const int32_t* positions, int n,
                             dec_stream_t stream) {
  if (int rc = rows_check(c, layer, type, seqs, n)) return rc;
  if (n == 0) return DEC_OK;
  return rows_call<false>(c, layer, const_cast<void*>(k), const_cast<void*>(v), type, row_stride, seqs, positions, n,
                          nullptr, stream);
}

extern "C" int dec_kv_read(const dec_kv_cache* c, int layer, void* k, void* v, int type, int64_t row_stride,
                           const int32_t* seqs, const int32_t* positions, int n, dec_stream_t stream) {
  if (int rc = rows_check(c, layer, type, seqs, n)) return rc;
  if (n == 0) return DEC_OK;
  return rows_call<true>(c, layer, k, v, type, row_stride, seqs, positions, n, nullptr, stream);
}

extern "C" int dec_kv_append_rotated(const dec_kv_cache* c, int layer, const dec_rope* rope, const void* q, void* q_out,
                                     int64_t q_stride, int64_t q_out_stride, int n_q_heads, const void* k, const void* v,
                                     int type, int64_t row_stride, const int32_t* seqs, const int32_t* positions, int n,
                                     dec_stream_t stream) {
  if (int rc = rows_check(c, layer, type, seqs, n)) return rc;
  if (int rc = rope_check(rope)) return rc;
  if (rope->head_dim != c->head_dim)
    return fail_no_handle(DEC_ERR_SHAPE, "a rotation of head_dim %d for a cache of %d", rope->head_dim, c->head_dim);
  if (n_q_heads < 0 || n_q_heads > 65536 || (int64_t)n * n_q_heads > (int64_t)1 << 30)
    return fail_no_handle(DEC_ERR_SHAPE, "%d rows of %d query heads (0..65536, and at most 2^30 in all)", n, n_q_heads);
  if (n == 0) return DEC_OK;
  RopeRows rows{};
  rows.r = rope_view(*rope, false);
  if (n_q_heads) {
    if (int rc = rope_rows_check(rope, q, q_out, type, q_stride, q_out_stride, n, n_q_heads, false, &rows)) return rc;
  }
  return rows_call<false>(c, layer, const_cast<void*>(k), const_cast<void*>(v), type, row_stride, seqs, positions, n,
                          &rows, stream);
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
