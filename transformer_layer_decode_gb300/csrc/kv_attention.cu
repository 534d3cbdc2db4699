// dec_kv_attention: attention of one query per sequence over a paged key/value
// cache, bf16 or in 4-bit blocks, with a sliding window and first rows that
// stay visible.
#include <atomic>
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "kv.h"

using namespace tld;

namespace {

// ---- shape of the launch ------------------------------------------------------
// A tile is 16 rows of one sequence and KV head; pages hold whole tiles.  A
// unit is (query, KV head, up to 8 of its query heads).  All visible tiles of
// all units, in that order, are one line that is cut evenly among the CTAs, by
// the lengths on the device: a long sequence is spread over many CTAs, short
// ones share one, and a captured graph follows the lengths.  Within a CTA the
// warps take tiles in turn, each with its own running softmax.  (Against a CTA
// per unit: a batch of ragged lengths waits for its longest, and one stream
// leaves most SMs idle.)
//
// What bounds it: bf16 pages, HBM: 46 windowed queries of 32 heads of 128, 1.46
// GB, take 222 us, 0.98 of the copy rate (7 queries of up to 24 001 rows, 1.15 GB:
// 175 us, 0.98; fp32 results 186, 0.92; head_dim 64 0.89).  4-bit pages, the
// latency of dependent steps, see WarpQ4: 24 queries of up to 24 001 rows, 1.54 GB,
// 315 us, 0.73; fp32 results 506, 0.45; head_dim 64 0.58 and 0.42.  A smaller batch,
// besides, the search for shares, a chain of loads and a merge per unit, and the
// joining launch, 10 to 20 us: 8 queries of up to 4096 rows 65 us for 366 MB of bf16
// pages, 35 us for 103 MB of 4-bit ones.  A short call, a chain of loads: one query of
// 127 rows 4.7 us where no sequence can be long, 6.9 in a table with room for 4096
// rows (counted, and a joining launch that finds nothing); of 8196 rows cut into 344
// parts 12.8 us, of which joining them takes 3.
constexpr int kTileRows = 16;
constexpr int kWarps = 4;
constexpr int kThreadsA = kWarps * 32;
constexpr int kHeadBlock = 8;      // query heads of a unit: the n of the tensor-core products
constexpr int kMaxQueries = 65536;
constexpr int kChunkRows = 128;    // queries whose tiles one warp counts at a time
constexpr int kMaxChunks = (kMaxQueries + kChunkRows - 1) / kChunkRows;
// A reference moves only when a score passes it by this (log2 units).
constexpr float kSlack = 5.f;

template <int D, bool Q4>
struct Tile {
  static constexpr int NB = D / 32;                                  // blocks of 32 dimensions
  static constexpr int kRowBytes = Q4 ? D / 2 : 2 * D;               // codes or values
  static constexpr int kHalf = kTileRows * (kRowBytes + (Q4 ? 2 * NB : 0));  // K or V, scales after the rows
  static constexpr int kBytes = 2 * kHalf;
  static constexpr int kStep = Q4 ? 2 : 1;                           // tiles a warp takes at a time
  static constexpr int kStages = Q4 ? (D == 128 ? 2 : 4) : (D == 128 ? 2 : 4);  // steps in its ring
  static constexpr int kSlot = kStep * kBytes;
  static constexpr int kRing = kWarps * kStages * kSlot;
  static constexpr int kMergeRow = D + 8;                            // floats; heads apart by 8 banks
  static constexpr int kMerge = kWarps * kHeadBlock * kMergeRow * 4; // the warps' sums, once the ring is drained
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
  static constexpr int kCtasPerSm = 3;
  // What a unit costs a CTA besides its tiles (page numbers, q, the sums of the
  // warps: about 2.5 us), in tiles; the tiles up to which a unit is not cut
  // between CTAs; and those up to which, if none can have more, every unit is
  // left to one CTA and nothing is counted.
  static constexpr int kUnit = Q4 ? 24 : 12, kShort = Q4 ? 40 : 20, kWhole = Q4 ? 48 : 24;
};

struct KvAttnParams {
  KvView c;
  const void* q;
  void* o;
  int64_t q_stride, o_stride;
  const int32_t* seqs;
  int n, nq, window, sinks;
  int group, head_blocks;  // query heads of a KV head, and blocks of 8 of them
  float scale;             // times log2(e)
  float* rec;              // [2 * CTAs][8][D]: sums of units cut between CTAs
  float2* ref;             // [2 * CTAs][8]: reference and sum of the weights
  int4* cut;               // [CTAs]: query, unit, CTA where it begins, CTAs that it goes on for
  int ctas;
  int cut_by_unit;         // cut is indexed by unit (there are no more of them than CTAs), not by CTA
};

// A query's visible rows: [0, first) and [lo, len).
struct Rows {
  int seq, len, lo, first;
  int sink_tiles, win_tile0, tiles;
};

__device__ __forceinline__ Rows query_rows(const KvAttnParams& p, int r, bool* bad) {
  Rows v{-1, 0, 0, 0, 0, 0, 0};
  const int s = p.seqs ? p.seqs[r] : r;
  if (s < 0) return v;
  const int len = s < p.c.n_seqs ? p.c.lens[s] : -1;
  if (len < 0 || len > p.c.max_pages * p.c.page_rows) {
    *bad = true;
    return v;
  }
  v.seq = s;
  v.len = len;
  v.lo = p.window && len > p.window ? len - p.window : 0;
  v.first = min(p.sinks, v.lo);
  v.sink_tiles = (v.first + kTileRows - 1) / kTileRows;
  v.win_tile0 = max(v.lo / kTileRows, v.sink_tiles);
  v.tiles = v.sink_tiles + (len + kTileRows - 1) / kTileRows - v.win_tile0;
  return v;
}

__device__ __forceinline__ int tile_row(const Rows& v, int t) {
  return kTileRows * (t < v.sink_tiles ? t : v.win_tile0 + t - v.sink_tiles);
}

// ---- tensor-core products and conversions ---------------------------------------
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }

// 1 / x of a power of two (2^-126 to 2^126).
__device__ __forceinline__ float inverse2(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

// Takes the next piece off (x, y): the pair rounded to 16 bits, leaving the rest.
__device__ __forceinline__ uint32_t take_bf16(float& x, float& y) {
  const uint32_t w = pack_bf16(x, y);
  x -= bf16lo(w);
  y -= bf16hi(w);
  return w;
}
__device__ __forceinline__ uint32_t take_f16(float& x, float& y) {
  const uint32_t w = pack_f16(x, y);
  const float2 f = unpack_f16(w);
  x -= f.x;
  y -= f.y;
  return w;
}

// Copies N bytes, of which the first `bytes` (N, or 0) from src and zeros for the rest.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int bytes) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Byte of 16-byte piece `piece` of row `row` within K or V of a staged tile.
// The pieces are placed so that the reads below touch every bank once: the K
// reads of 8 lanes (rows 2i, 2i + 1, four neighbouring pieces each) and the V
// reads (rows 0, 2, 4, 6 or 1, 3, 5, 7, the same pieces of each).
template <int D, bool Q4>
__device__ __forceinline__ int staged(int row, int piece) {
  const int j = row & 7, t = j >> 1;
  if constexpr (!Q4) {  // rows of 128 or 256 bytes
    return row * (2 * D) + ((piece ^ ((t ^ ((j & 1) << 1)) << 1)) << 4);
  } else if constexpr (D == 128) {  // rows of 64 bytes, two to a line of banks
    return (row >> 1) * 128 + (((j & 1) ^ (t & 1)) << 6) + ((piece ^ (t & 2)) << 4);
  } else {  // rows of 32 bytes, four to a line
    return (row >> 3) * 256 + ((j & 1) << 7) + ((t ^ ((j & 1) << 1)) << 5) + (piece << 4);
  }
}

// ---- the warp's part: tiles of one unit -------------------------------------------
// For one tile the scores are computed as S[head][row] = q K^T: q is the
// 16-row operand (its 8 heads in rows 0-7; rows 8-15 hold the next piece of the
// same heads, so that 16-bit products add up to fp32 ones), K the other, 8 rows
// of the tile at a time.  Lane (g, t) = (lane / 4, lane % 4) then has head g and
// rows 2t, 2t + 1 of each half, which is exactly the operand P^T of the second
// product, O^T[dim][head] = V^T P^T: no value changes lanes.  The order of the
// dimensions within a product and of O's rows is free, and chosen so that a
// lane's operands are whole words of the staged rows.
//
// The softmax runs on a reference that moves only when a score passes it by
// kSlack: the weights are 2^(score - ref), their sum l and the outputs follow
// it, and o / l does not depend on it.
template <int D>
struct WarpSums {
  static constexpr int NB = D / 32;
  float acc[NB][2][4];  // O^T: [0..1] a dimension (out_dim) of heads 2t, 2t + 1; [2..3] the next dimension

  __device__ __forceinline__ void clear_acc() {
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[x][y][i] = 0.f;
  }

  // The tensor cores cut sums off rather than round them: over a long sequence of
  // values with a mean an accumulator there would fall short by up to 2^-24 a
  // product (1.2e-5 of the result for 24 sequences of 24000 rows).  For fp32 results
  // a tile's products are summed apart, and added here, rounded to the nearest: 8 % of
  // the time over 4-bit pages (374 and 405 us where nothing else differed), 2 % of a
  // short call.
  __device__ __forceinline__ void add_tile(float (&to)[4], const float (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] += o[i];
  }

  __device__ __forceinline__ void scale_block(int x, float k) {
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[x][y][i] *= k;
  }

  __device__ __forceinline__ void scale_acc(float k0, float k1) {
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) acc[x][y][0] *= k0, acc[x][y][1] *= k1, acc[x][y][2] *= k0, acc[x][y][3] *= k1;
  }
};

// The softmax state of a lane that has the scores of head g.
template <int D>
struct WarpHead : WarpSums<D> {
  float ref, l;

  __device__ __forceinline__ void clear() {
    this->clear_acc();
    ref = -3e38f;
    l = 0.f;
  }

  // Moves every head's reference so that its largest score (mx: the largest of
  // this lane's new ones) has the weight 2^lift.
  __device__ __forceinline__ void raise(float mx, float lift) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float now = fmaxf(ref, mx - lift);
    const float keep = exp2_approx(ref - now);
    ref = now;
    l *= keep;
    const int t = threadIdx.x & 3;
    this->scale_acc(__shfl_sync(0xffffffffu, keep, 8 * t), __shfl_sync(0xffffffffu, keep, 8 * t + 4));
  }

  __device__ __forceinline__ void write_refs(float2* to, int lane) {
    float sum = l;
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if ((lane & 3) == 0) to[lane >> 2] = make_float2(ref, sum);
  }
};

// The same of a lane that has the scores of heads 2t and 2t + 1.
template <int D>
struct WarpHeadPair : WarpSums<D> {
  float ref[2], l[2];

  __device__ __forceinline__ void clear() {
    this->clear_acc();
    ref[0] = ref[1] = -3e38f;
    l[0] = l[1] = 0.f;
  }

  __device__ __forceinline__ void raise(float mx0, float mx1, float lift) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
    }
    const float now0 = fmaxf(ref[0], mx0 - lift), now1 = fmaxf(ref[1], mx1 - lift);
    const float keep0 = exp2_approx(ref[0] - now0), keep1 = exp2_approx(ref[1] - now1);
    ref[0] = now0, ref[1] = now1;
    l[0] *= keep0, l[1] *= keep1;
    this->scale_acc(keep0, keep1);
  }

  __device__ __forceinline__ void write_refs(float2* to, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane < 4) to[2 * lane + i] = make_float2(ref[i], sum);
    }
  }
};

// Of a tile's 16 rows the lane's four: bit i is row (i & 1) + 2t + 8 (i >> 1).
__device__ __forceinline__ uint32_t rows_of_lane(uint32_t rows, int t) {
  const uint32_t r = rows >> (2 * t);
  return (r & 3) | (r >> 6 & 12);
}

// Eight dimensions 32 b + 8 t .. of a query as fp32.
template <int NB, class T>
__device__ __forceinline__ void load_query(const T* q, bool valid, int t, float (&x)[NB][8]) {
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (!valid) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[b][i] = 0.f;
    } else if constexpr (sizeof(T) == 4) {
      const float4* p = reinterpret_cast<const float4*>(q + 32 * b + 8 * t);
      const float4 u = p[0], w = p[1];
      x[b][0] = u.x, x[b][1] = u.y, x[b][2] = u.z, x[b][3] = u.w;
      x[b][4] = w.x, x[b][5] = w.y, x[b][6] = w.z, x[b][7] = w.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(q + 32 * b + 8 * t);
      x[b][0] = bf16lo(u.x), x[b][1] = bf16hi(u.x), x[b][2] = bf16lo(u.y), x[b][3] = bf16hi(u.y);
      x[b][4] = bf16lo(u.z), x[b][5] = bf16hi(u.z), x[b][6] = bf16lo(u.w), x[b][7] = bf16hi(u.w);
    }
  }
}

// bf16 pages.  fp32 calls take q and the weights in three bf16 pieces (24
// bits); bf16 calls take q as it is and the weights in two (16 bits, against
// the 8 of their results).
template <int D, class T>
struct WarpBf16 : WarpHead<D> {
  using Sums = WarpSums<D>;
  static constexpr int NB = Sums::NB, kPieces = sizeof(T) == 4 ? 3 : 2;
  static constexpr bool kWhole = sizeof(T) == 2;  // q is one piece
  uint32_t a[2 * NB][4];                // q: the first two pieces
  uint32_t a3[kWhole ? 1 : 2 * NB][2];  // the third
  float f;                              // score = f * product, in log2 units

  __device__ static int out_dim(int x, int y, int g) { return 64 * (x >> 1) + 8 * g + 4 * (x & 1) + 2 * y; }
  __device__ __forceinline__ float out_unit(int) const { return 1.f; }

  __device__ __forceinline__ void set_q(float (&x)[NB][8], int, float scale) {
    f = scale;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t(&w)[4] = a[2 * b + h];
        float(&y)[8] = x[b];
        w[0] = take_bf16(y[4 * h], y[4 * h + 1]);
        w[2] = take_bf16(y[4 * h + 2], y[4 * h + 3]);
        if constexpr (kWhole) {
          w[1] = w[3] = 0;
        } else {
          w[1] = take_bf16(y[4 * h], y[4 * h + 1]);
          w[3] = take_bf16(y[4 * h + 2], y[4 * h + 3]);
          a3[2 * b + h][0] = pack_bf16(y[4 * h], y[4 * h + 1]);
          a3[2 * b + h][1] = pack_bf16(y[4 * h + 2], y[4 * h + 3]);
        }
      }
    this->clear();
  }

  // One staged tile.  EDGE: some row is not visible; rows_seen: a bit for each that is.
  template <bool EDGE>
  __device__ __forceinline__ void step(const uint8_t* st, int lane, uint64_t rows_seen) {
    using L = Tile<D, false>;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t seen = rows_of_lane((uint32_t)rows_seen, t);
    const uint8_t* sv = st + L::kHalf;
    float s[4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float c[4] = {0.f, 0.f, 0.f, 0.f}, low[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(st + staged<D, false>(8 * b + g, 4 * j + t));
        mma_bf16(c, a[2 * j][0], a[2 * j][1], a[2 * j][2], a[2 * j][3], w.x, w.y);
        if constexpr (!kWhole) mma_bf16(low, a3[2 * j][0], 0, a3[2 * j][1], 0, w.x, w.y);
        mma_bf16(c, a[2 * j + 1][0], a[2 * j + 1][1], a[2 * j + 1][2], a[2 * j + 1][3], w.z, w.w);
        if constexpr (!kWhole) mma_bf16(low, a3[2 * j + 1][0], 0, a3[2 * j + 1][1], 0, w.z, w.w);
      }
      s[2 * b] = (kWhole ? c[0] : c[0] + (c[2] + low[0])) * f;
      s[2 * b + 1] = (kWhole ? c[1] : c[1] + (c[3] + low[1])) * f;
    }
    if (EDGE) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(seen >> i & 1)) s[i] = -INFINITY;
    }
    const float mx = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
    if (__any_sync(0xffffffffu, mx > this->ref + kSlack)) this->raise(mx, 0.f);
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = exp2_approx(s[i] - this->ref);
    this->l += (w[0] + w[1]) + (w[2] + w[3]);
    uint32_t pw[kPieces][2];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) pw[k][0] = take_bf16(w[0], w[1]), pw[k][1] = take_bf16(w[2], w[3]);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = *reinterpret_cast<const uint4*>(sv + staged<D, false>((i & 1) + 2 * t + 8 * (i >> 1), 8 * c + g));
        if (EDGE && !(seen >> i & 1)) v[i] = make_uint4(0, 0, 0, 0);  // 0 * NaN would be NaN
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = k == 0 ? v[i].x : k == 1 ? v[i].y : k == 2 ? v[i].z : v[i].w;
        const uint32_t a0 = __byte_perm(r[0], r[1], 0x5410), a1 = __byte_perm(r[0], r[1], 0x7632);
        const uint32_t a2 = __byte_perm(r[2], r[3], 0x5410), a3_ = __byte_perm(r[2], r[3], 0x7632);
        if constexpr (kWhole) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
            mma_bf16(this->acc[2 * c + (k >> 1)][k & 1], a0, a1, a2, a3_, pw[i][0], pw[i][1]);
        } else {  // (see add_tile)
          float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = kPieces - 1; i >= 0; --i) mma_bf16(o, a0, a1, a2, a3_, pw[i][0], pw[i][1]);
          this->add_tile(this->acc[2 * c + (k >> 1)][k & 1], o);
        }
      }
    }
  }
};

// 4-bit pages.  What bounds it is the work on a row, not HBM: a row of 128
// dimensions is 144 bytes for K and V, 1/3.6 of the bf16 row with the same
// number of values.  So the codes enter the products with as little unpacking
// as can be exact.
//  - K, bf16 results: a nibble n where it lies in a 16-bit word is the fp16 number
//    n 2^-24, or n 2^-20 four bits up (against q / 16): an AND, no conversion.  The
//    8 that codes are stored with is taken off by one more product per 16 rows, of
//    the block scales with -8 * (sum of q over the block).  The tensor cores align
//    such small numbers by fp16's smallest exponent and cut off what is then below
//    the sum's last bit: scores are off by 4e-7 of themselves.
//  - V, and K for fp32 results: 1024 + n or 1024 + 16 n by an OR, and n - 8 by one
//    addition or FMA (K's as subnormals took 7 % less time: 405 and 431 us).
//  - K's block scales multiply the fp32 sums over a block, V's the weights.
// q is scaled by a power of two and taken in two fp16 pieces (22 bits; bf16 q
// needs one), and so is weight * scale for fp32 results; for bf16 results it
// is one fp16 number (11 bits, against the 8 of the results).  With one piece
// each, the scores are computed the other way round, S^T = K q^T, 16 rows at a
// time, which takes half the products and block scales, and the weights, packed
// in pairs of heads, are turned by movmatrix.  Per tile of 16 rows of 128
// dimensions this takes 345 instructions, 170 of them on the integer pipe (two
// cycles each), and 155 cycles of an SM, whose share of HBM would take 101 for the
// tile's bytes.  No pipe is full in them: issue is active in 56 %, the integer pipe
// in 55.  Three warps a scheduler (168 registers) each go through scores, maximum,
// exponentials and V's products one after another, and wait for each.  fp32 results
// take 614 instructions and 245 cycles, with issue active in 63 %: two sets of
// products, K's codes made normal numbers, the second pieces and their 2^kLow (8 %).
// Two tiles a step: one takes 12 % longer (its loop and its checks), four win
// 5 % on long sequences and lose 40 % on batches of short ones.
template <int D, class T>
struct WarpQ4 : std::conditional_t<sizeof(T) == 2, WarpHeadPair<D>, WarpHead<D>> {
  using Sums = WarpSums<D>;
  using L = Tile<D, true>;
  static constexpr int NB = Sums::NB, kTiles = L::kStep;
  static constexpr bool kWhole = sizeof(T) == 2;  // q, and the weights, are one piece
  // The largest weight enters its products as 2^9 to 2^(9 + kSlack), so that they,
  // with scales below one, fit fp16 and the others are well above its smallest step.
  // kWhole has these 9 in the exponential; fp32 results have them in `unit`: an
  // exponent near 9 is good to 2^-21, one near 0 to much more.  The scales of a block
  // are brought below one by a power of two of their own: the blocks of a row can
  // differ by as much as fp16 does, and a product's step should be that of its block.
  // The second piece of a product enters times 2^kLow, which comes off its sums: it is
  // the first one's rounding, 2^-11 of it, and would lose its bits to fp16's smallest
  // step where the product is below 2^-3.
  static constexpr int kRoom = 9, kLow = 11;
  static constexpr float kLift = kWhole ? kRoom : 0;
  uint32_t a[2 * NB][kWhole ? 2 : 4];  // q
  uint32_t bias[kWhole ? 2 : 1];       // kWhole: -8 sum of q per block, in three pieces: operand of one product
  float f, f1;                         // score = f * product, in log2 units; kWhole: f of head 2t, f1 of the next
  float top0, top1;                    // V scales seen in the two blocks that this lane looks at are below 2^e
  float unit[kWhole ? 1 : NB];         // a block's enter times 2^(kRoom - e); kWhole: in unit2, as far as fp16 goes 2^-e, or
  __half2 unit2[kWhole ? NB / 2 : 1];  // as they are for e in [-2, 0] (e = -1 is usual; scaling costs 2 %)
  bool scaled;                         // kWhole: some block's are not as they are

  __device__ static int out_dim(int x, int y, int g) { return 32 * x + 4 * g + 2 * y; }
  __device__ __forceinline__ float unit_of(int x) const {
    if constexpr (kWhole) return x & 1 ? __high2float(unit2[x >> 1]) : __low2float(unit2[x >> 1]);
    else return unit[x];
  }
  __device__ __forceinline__ float out_unit(int x) const { return inverse2(unit_of(x)); }

  __device__ __forceinline__ void set_q(float (&x)[NB][8], int t, float scale) {
    float mx = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[b][i]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = (int)(__float_as_uint(mx) >> 23) - 126;  // mx < 2^e
    const int sh = min(14 - e, 120);                       // q to below 2^14
    const float up = __uint_as_float((uint32_t)(127 + max(sh, -120)) << 23);
    f = scale * __uint_as_float((uint32_t)(127 + (kWhole ? min(24 - sh, 127) : -sh)) << 23);
    if (!(mx < INFINITY)) f = __uint_as_float(0x7fffffffu);  // an infinity in q: NaN
    float sums[NB];  // kWhole: of q
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[b][i] *= up;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t(&w)[kWhole ? 2 : 4] = a[2 * b + h];
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
          const float part = kWhole && odd ? 1.f / 16 : 1.f;
          float y0 = x[b][2 * h + odd] * part, y1 = x[b][4 + 2 * h + odd] * part;
          const uint32_t hi = take_f16(y0, y1), lo = pack_f16(y0, y1);
          if constexpr (kWhole) {  // (lo is zero)
            const float2 u = unpack_f16(hi);
            w[odd] = hi;
            sum += (u.x + u.y) * (odd ? 16.f : 1.f);
          } else {
            w[2 * odd] = hi;
            w[2 * odd + 1] = lo;
          }
        }
      }
      if constexpr (kWhole) {
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sums[b] = sum * (-8.f / (1 << 10));  // (times 2^14: the codes' 2^-24 in fp16's range)
      }
    }
    if constexpr (kWhole) {
      uint32_t piece[3][NB / 2];
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < NB / 2; ++j) piece[k][j] = take_f16(sums[2 * j], sums[2 * j + 1]);
      // the 16 entries of a row of the operand: piece by piece, the blocks in order; then zeros
      if constexpr (NB == 4) {
        bias[0] = t == 0 ? piece[0][0] : t == 1 ? piece[0][NB / 2 - 1] : t == 2 ? piece[1][0] : piece[1][NB / 2 - 1];
        bias[1] = t == 0 ? piece[2][0] : t == 1 ? piece[2][NB / 2 - 1] : 0;
      } else {
        bias[0] = t == 0 ? piece[0][0] : t == 1 ? piece[1][0] : t == 2 ? piece[2][0] : 0;
        bias[1] = 0;
      }
      f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
      f = __shfl_sync(0xffffffffu, f, 8 * t);
    }
    this->clear();
    top0 = top1 = 5.9604644775390625e-8f;  // fp16's smallest: a scale that is not 0 reaches it
    if constexpr (kWhole) {
#pragma unroll
      for (int j = 0; j < NB / 2; ++j) unit2[j] = __float2half2_rn(1.f);
    } else {
#pragma unroll
      for (int j = 0; j < NB; ++j) unit[j] = 1.f;
    }
    scaled = false;
  }

  // Makes room for V scales up to s0 and s1 in this lane's two blocks, which are 2 i
  // and 2 i + 1 for i = lane % (NB / 2).
  __device__ __forceinline__ void make_room(float s0, float s1) {
#pragma unroll
    for (int o = NB / 2; o < 32; o <<= 1) {
      s0 = fmaxf(s0, __shfl_xor_sync(0xffffffffu, s0, o));
      s1 = fmaxf(s1, __shfl_xor_sync(0xffffffffu, s1, o));
    }
    auto above = [](float s, float top) {  // the next power of two (-23 <= e <= 16)
      return s < top ? top : __uint_as_float(((__float_as_uint(s) >> 23) + 1) << 23);
    };
    top0 = above(s0, top0);
    top1 = above(s1, top1);
    scaled = false;
    float now[NB];
#pragma unroll
    for (int x = 0; x < NB; ++x) {
      const float top = __shfl_sync(0xffffffffu, x & 1 ? top1 : top0, x >> 1);
      const int e = (int)(__float_as_uint(top) >> 23) - 127;
      const bool fits = kWhole && e <= 0 && e >= -2;
      now[x] = __uint_as_float((uint32_t)(127 + (kWhole ? (fits ? 0 : -max(e, -15)) : kRoom - e)) << 23);
      scaled |= now[x] != 1.f;
      this->scale_block(x, now[x] * out_unit(x));
    }
    if constexpr (kWhole) {
#pragma unroll
      for (int j = 0; j < NB / 2; ++j) unit2[j] = __floats2half2_rn(now[2 * j], now[2 * j + 1]);
    } else {
#pragma unroll
      for (int x = 0; x < NB; ++x) unit[x] = now[x];
    }
  }

  // kTiles staged tiles.  EDGE: some row is not visible; rows_seen: a bit for each that is.
  template <bool EDGE>
  __device__ __forceinline__ void step(const uint8_t* st, int lane, uint64_t rows_seen) {
    const int g = lane >> 2, t = lane & 3;
    const __half2 m1032 = __float2half2_rn(-1032.f), sixteenth = __float2half2_rn(0.0625f), m72 = __float2half2_rn(-72.f);
    // n - 8 of the nibbles 0 and 4, or 1 and 5, of a word
    auto low = [&](uint32_t z) {
      const uint32_t u = (z & 0x000f000fu) | 0x64006400u;  // 1024 + n
      const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&u), m1032);
      return *reinterpret_cast<const uint32_t*>(&r);
    };
    auto high = [&](uint32_t z) {
      const uint32_t u = (z & 0x00f000f0u) | 0x64006400u;  // 1024 + 16 n
      const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&u), sixteenth, m72);
      return *reinterpret_cast<const uint32_t*>(&r);
    };
    // scores: of head g, rows 2t, 2t + 1 of each half; kWhole: of heads 2t, 2t + 1, rows g and g + 8
    float s[4 * kTiles];
    __half2 most = __float2half2_rn(0.f);  // the largest of V's scales, between the lanes
#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
      const uint8_t* sk = st + k * L::kBytes;
      const uint8_t* ks_at = sk + kTileRows * L::kRowBytes;
      if (D == 128 || lane < 16) {
        __half2 h = *reinterpret_cast<const __half2*>(ks_at + L::kHalf + 4 * lane);
        if (EDGE && !(rows_seen >> (16 * k + lane / (NB / 2)) & 1)) h = __float2half2_rn(0.f);
        most = __hmax2(most, __habs2(h));
      }
      uint32_t w[2][NB];  // rows g, g + 8: blocks 0, 1 (and 2, 3) of dimension groups 2t, then of 2t + 1
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(sk + staged<D, true>(8 * b + g, t));
          w[b][0] = u.x, w[b][1] = u.y, w[b][2] = u.z, w[b][3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(sk + staged<D, true>(8 * b + g, t >> 1) + 8 * (t & 1));
          w[b][0] = u.x, w[b][1] = u.y;
        }
      }
      auto codes = [&](int b, int j) {  // four of group 2t, four of 2t + 1
        return __byte_perm(w[b][j >> 1], w[b][NB / 2 + (j >> 1)], j & 1 ? 0x7632 : 0x5410);
      };
      if constexpr (kWhole) {
        uint32_t ks[2][NB / 2];  // K's scales of rows g, g + 8
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if constexpr (D == 128) {
            const uint2 u = *reinterpret_cast<const uint2*>(ks_at + 64 * b + 8 * g);
            ks[b][0] = u.x, ks[b][NB / 2 - 1] = u.y;
          } else {
            ks[b][0] = *reinterpret_cast<const uint32_t*>(ks_at + 32 * b + 4 * g);
          }
        }
        const uint32_t odd = (uint32_t) - (t & 1);  // the blocks of this lane's part of the bias
        const uint32_t z0 = (ks[0][0] & ~odd) | (ks[0][NB / 2 - 1] & odd), z1 = (ks[1][0] & ~odd) | (ks[1][NB / 2 - 1] & odd);
        float z[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(z, z0, z1, z0, z1, bias[0], bias[1]);
        float r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = z[i] * (1.f / (1 << 14));
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t x0 = codes(0, j), x1 = codes(1, j), y0 = x0 >> 8, y1 = x1 >> 8;
          mma_f16(c, x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, a[2 * j][0], a[2 * j][1]);
          mma_f16(c, y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u, a[2 * j + 1][0],
                  a[2 * j + 1][1]);
          const float2 u0 = unpack_f16(ks[0][j >> 1]), u1 = unpack_f16(ks[1][j >> 1]);
          const float k0 = j & 1 ? u0.y : u0.x, k1 = j & 1 ? u1.y : u1.x;
          r[0] = fmaf(k0, c[0], r[0]);
          r[1] = fmaf(k0, c[1], r[1]);
          r[2] = fmaf(k1, c[2], r[2]);
          r[3] = fmaf(k1, c[3], r[3]);
        }
        s[4 * k] = r[0] * f;
        s[4 * k + 1] = r[1] * f1;
        s[4 * k + 2] = r[2] * f;
        s[4 * k + 3] = r[3] * f1;
        if (EDGE) {
          if (!(rows_seen >> (16 * k + g) & 1)) s[4 * k] = s[4 * k + 1] = -INFINITY;
          if (!(rows_seen >> (16 * k + 8 + g) & 1)) s[4 * k + 2] = s[4 * k + 3] = -INFINITY;
        }
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          __half2 ks[2][NB / 2];
          if constexpr (D == 128) *reinterpret_cast<uint4*>(ks) = *reinterpret_cast<const uint4*>(ks_at + 64 * b + 16 * t);
          else *reinterpret_cast<uint2*>(ks) = *reinterpret_cast<const uint2*>(ks_at + 32 * b + 8 * t);
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t x = codes(b, j), y = x >> 8;
            mma_f16(c, a[2 * j][0], a[2 * j][1], a[2 * j][2], a[2 * j][3], low(x), high(x));
            mma_f16(c, a[2 * j + 1][0], a[2 * j + 1][1], a[2 * j + 1][2], a[2 * j + 1][3], low(y), high(y));
            const float k0 = __half2float(j & 1 ? __high2half(ks[0][j >> 1]) : __low2half(ks[0][j >> 1]));
            const float k1 = __half2float(j & 1 ? __high2half(ks[1][j >> 1]) : __low2half(ks[1][j >> 1]));
            s0 = fmaf(k0, c[0] + c[2], s0);
            s1 = fmaf(k1, c[1] + c[3], s1);
          }
          s[4 * k + 2 * b] = s0 * f;
          s[4 * k + 2 * b + 1] = s1 * f;
        }
        if (EDGE) {
          const uint32_t seen = rows_of_lane((uint32_t)(rows_seen >> (16 * k)) & 0xffff, t);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(seen >> i & 1)) s[4 * k + i] = -INFINITY;
        }
      }
    }
    const float most0 = __low2float(most), most1 = __high2float(most);
    const bool over = most0 >= top0 || most1 >= top1;
    float w[4 * kTiles];
    if constexpr (kWhole) {
      float mx0 = fmaxf(s[0], s[2]), mx1 = fmaxf(s[1], s[3]);
#pragma unroll
      for (int i = 4; i < 4 * kTiles; i += 2) mx0 = fmaxf(mx0, s[i]), mx1 = fmaxf(mx1, s[i + 1]);
      if (__any_sync(0xffffffffu,
                     mx0 > this->ref[0] + (kLift + kSlack) || mx1 > this->ref[1] + (kLift + kSlack) || over)) {
        if (__any_sync(0xffffffffu, over)) make_room(most0, most1);
        this->raise(mx0, mx1, kLift);
      }
#pragma unroll
      for (int i = 0; i < 4 * kTiles; ++i) {
        w[i] = exp2_approx(s[i] - this->ref[i & 1]);
        this->l[i & 1] += w[i];
      }
    } else {
      float mx = s[0];
#pragma unroll
      for (int i = 1; i < 4 * kTiles; ++i) mx = fmaxf(mx, s[i]);
      if (__any_sync(0xffffffffu, mx > this->ref + (kLift + kSlack) || over)) {
        if (__any_sync(0xffffffffu, over)) make_room(most0, most1);
        this->raise(mx, kLift);
      }
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * kTiles; ++i) {
        w[i] = exp2_approx(s[i] - this->ref);
        sum += w[i];
      }
      this->l += sum;
    }

#pragma unroll
    for (int k = 0; k < kTiles; ++k) {
      const uint8_t* sv = st + k * L::kBytes + L::kHalf;
      const uint8_t* vs_at = sv + kTileRows * L::kRowBytes;
      __half2 vs[4][NB / 2];  // V's scales of the lane's rows
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if constexpr (D == 128)
          *reinterpret_cast<uint4*>(vs[2 * b]) = *reinterpret_cast<const uint4*>(vs_at + 64 * b + 16 * t);
        else *reinterpret_cast<uint2*>(vs[2 * b]) = *reinterpret_cast<const uint2*>(vs_at + 32 * b + 8 * t);
      }
      if (EDGE) {  // 0 * NaN would be NaN
        const uint32_t seen = rows_of_lane((uint32_t)(rows_seen >> (16 * k)) & 0xffff, t);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(seen >> i & 1)) {
#pragma unroll
            for (int j = 0; j < NB / 2; ++j) vs[i][j] = __float2half2_rn(0.f);
          }
      }
      if constexpr (kWhole) {
        if (scaled) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NB / 2; ++j) vs[i][j] = __hmul2(vs[i][j], unit2[j]);
        }
      }
      uint32_t v[4][NB / 2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (i & 1) + 2 * t + 8 * (i >> 1);
        if constexpr (D == 128) {
          const uint2 u = *reinterpret_cast<const uint2*>(sv + staged<D, true>(row, g >> 1) + 8 * (g & 1));
          v[i][0] = u.x, v[i][1] = u.y;
        } else {
          v[i][0] = *reinterpret_cast<const uint32_t*>(sv + staged<D, true>(row, g >> 2) + 4 * (g & 3));
        }
      }
      uint32_t ph[2];
      if constexpr (kWhole) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          // row g + 8 b of heads 2t, 2t + 1 to rows 2t, 2t + 1 of that half of head g
          const uint32_t rows = pack_f16(w[4 * k + 2 * b], w[4 * k + 2 * b + 1]);
          asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(ph[b]) : "r"(rows));
        }
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        constexpr int kPieces = kWhole ? 1 : 2;
        uint32_t pw[kPieces][2];  // weight * scale: rows 2t, 2t + 1 of each half
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const __half2 h0 = vs[2 * b][j >> 1], h1 = vs[2 * b + 1][j >> 1];
          if constexpr (kWhole) {
            const __half2 both = j & 1 ? __highs2half2(h0, h1) : __lows2half2(h0, h1);
            const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&ph[b]), both);
            pw[0][b] = *reinterpret_cast<const uint32_t*>(&y);
          } else {
            float y0 = w[4 * k + 2 * b] * unit[j] * (j & 1 ? __high2float(h0) : __low2float(h0));
            float y1 = w[4 * k + 2 * b + 1] * unit[j] * (j & 1 ? __high2float(h1) : __low2float(h1));
            pw[0][b] = take_f16(y0, y1);
            pw[1][b] = pack_f16(y0 * (1 << kLow), y1 * (1 << kLow));
          }
        }
        uint32_t z0 = __byte_perm(v[0][j >> 1], v[1][j >> 1], j & 1 ? 0x7632 : 0x5410);
        uint32_t z1 = __byte_perm(v[2][j >> 1], v[3][j >> 1], j & 1 ? 0x7632 : 0x5410);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t a0 = low(z0), a1 = high(z0), a2 = low(z1), a3 = high(z1);
          if constexpr (kWhole) {
            mma_f16(this->acc[j][y], a0, a1, a2, a3, pw[0][0], pw[0][1]);
          } else {  // (see add_tile)
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(o, a0, a1, a2, a3, pw[kPieces - 1][0], pw[kPieces - 1][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= 1.f / (1 << kLow);
            mma_f16(o, a0, a1, a2, a3, pw[0][0], pw[0][1]);
            this->add_tile(this->acc[j][y], o);
          }
          z0 >>= 8;
          z1 >>= 8;
        }
      }
    }
  }
};

// Fills a stage with a tile: K's rows (Q4: codes) begin at `src`, their scales
// `scales` bytes behind, V's half_bytes behind K's; not `there`: with zeros.
template <int D, bool Q4>
__device__ __forceinline__ void stage_tile(uint32_t dst, const uint8_t* src, int scales, int64_t half_bytes, int lane,
                                           bool there) {
  using L = Tile<D, Q4>;
  constexpr int PPR = L::kRowBytes / 16, N = kTileRows * PPR / 32;
  const uint8_t* k = src + 16 * lane;
  const uint8_t* v = src + (half_bytes + 16 * lane);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = i * 32 + lane, to = staged<D, Q4>(at / PPR, at % PPR);
    cp_async<16>(dst + to, k + 512 * i, there ? 16 : 0);
    cp_async<16>(dst + L::kHalf + to, v + 512 * i, there ? 16 : 0);
  }
  if constexpr (Q4) {  // half the lanes K's scales, half V's
    constexpr int kPart = L::NB * 2;
    const int64_t from = (lane < 16 ? 0 : half_bytes) + (lane & 15) * kPart;
    const int to = kTileRows * L::kRowBytes + (lane < 16 ? 0 : L::kHalf) + (lane & 15) * kPart;
    cp_async<kPart>(dst + to, src + (from + scales), there ? kPart : 0);
  }
}

template <class T, int N>
__device__ __forceinline__ void store_out(T* p, const float (&x)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<uint2*>(p + i) = make_uint2(pack_bf16(x[i], x[i + 1]), pack_bf16(x[i + 2], x[i + 3]));
  }
}

// The sum over no weight is zero; NaN stays.
__device__ __forceinline__ float over(float l) { return l == 0.f ? 0.f : 1.f / l; }

// What a thread holds of a unit's sums over a CTA's tiles: N dimensions from e
// of head h, relative to the reference m, and the sum of the weights.
template <int D>
struct UnitSums {
  static constexpr int N = D / 16;
  float x[N], m, l;
};

// The CTA's sums over tiles t0 .. t1 - 1 of unit u of query r.
template <int D, bool Q4, class T>
__device__ __forceinline__ UnitSums<D> unit_sums(const KvAttnParams& p, const Rows& v, int r, int u, int t0, int t1,
                                                 uint8_t* smem) {
  using L = Tile<D, Q4>;
  using W = std::conditional_t<Q4, WarpQ4<D, T>, WarpBf16<D, T>>;
  constexpr int ST = L::kStages, kRound = kWarps * L::kStep;
  __shared__ float2 warp_ref[kWarps][kHeadBlock];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const KvView& c = p.c;
  const int head = u / p.head_blocks, h0 = (u % p.head_blocks) * kHeadBlock;
  const int n_heads = min(kHeadBlock, p.group - h0);
  __syncthreads();  // the sums of the unit before have been read

  // ---- the warp's tiles: kStep from t0 + warp * kStep, again kWarps * kStep further on, ...
  const int nt = (t1 - t0) / kRound * L::kStep + min(max((t1 - t0) % kRound - warp * L::kStep, 0), L::kStep);
  const uint32_t ring = smem_u32(smem) + warp * ST * L::kSlot;
  const int32_t* table = c.table + (int64_t)v.seq * c.max_pages;
  // K rows of a tile, and how far behind its scales are; -1: there is none
  unsigned long long cur_src = 0, nxt_src = 0;
  int cur_scales = -1, nxt_scales = -1;
  bool doubt = false;  // a tile had no page
  auto tile_no = [&](int i) { return t0 + warp * L::kStep + i / L::kStep * kRound + i % L::kStep; };
  auto page_of = [&](int row) {
    if (!KV_IN_BOUNDS(c, row >= 0 && row < c.max_pages * c.page_rows)) return -1;
    const int page = table[row / c.page_rows];
    return page >= 0 && page < c.n_pages ? page : -1;
  };
  auto fetch = [&](int i0) {  // where the warp's tiles i0 .. i0 + 31 lie, one per lane
    const int i = i0 + lane;
    nxt_src = reinterpret_cast<unsigned long long>(c.pool);
    nxt_scales = -1;
    if (i < nt) {
      const int at = tile_row(v, tile_no(i)), page = page_of(at), row = at % c.page_rows;
      if (page >= 0 && KV_IN_BOUNDS(c, row + kTileRows <= c.page_rows && head < c.nkv)) {
        nxt_src = reinterpret_cast<unsigned long long>(c.pool + page * c.page_bytes + head * c.head_bytes +
                                                       row * L::kRowBytes);
        nxt_scales = (c.page_rows - row) * L::kRowBytes + row * 2 * L::NB;
      } else {
        atomicOr(c.status, DEC_KV_BAD_INDEX);
        doubt = true;
      }
    }
  };
  auto issue = [&](int j, uint32_t dst) {
    if ((j & (32 / L::kStep - 1)) == 0) {
      cur_src = nxt_src;
      cur_scales = nxt_scales;
      fetch(j * L::kStep + 32);
      doubt = __any_sync(0xffffffffu, doubt);
    }
    if (j * L::kStep < nt && KV_IN_BOUNDS(c, dst >= smem_u32(smem) && dst + L::kSlot <= smem_u32(smem) + L::kRing)) {
#pragma unroll
      for (int k = 0; k < L::kStep; ++k) {
        const int i = (j * L::kStep + k) & 31;
        const unsigned long long src = __shfl_sync(0xffffffffu, cur_src, i);
        const int scales = __shfl_sync(0xffffffffu, cur_scales, i);
        stage_tile<D, Q4>(dst + k * L::kBytes, reinterpret_cast<const uint8_t*>(src), max(scales, 0), c.half_bytes, lane,
                          scales >= 0);
      }
    }
    cp_async_commit();
  };
  // the steps, from plain0 on for plain_n, whose every row is visible (those of the first rows aside)
  const int n0 = t0 + warp * L::kStep;
  const int full0 = v.sink_tiles + (v.win_tile0 * kTileRows < v.lo), full1 = v.sink_tiles + v.len / kTileRows - v.win_tile0;
  const int plain0 = full0 > n0 ? (full0 - n0 + kRound - 1) / kRound : 0;
  const int plain_n =
      min(nt / L::kStep, full1 - L::kStep >= n0 ? (full1 - L::kStep - n0) / kRound + 1 : 0) - plain0;
  const bool asks = g < n_heads && KV_IN_BOUNDS(c, r >= 0 && r < p.n && (int64_t)head * p.group + h0 + g < p.nq);
  float x[L::NB][8];  // q, read while the page numbers are, and made operands while the first tiles are under way
  load_query<L::NB>(
      static_cast<const T*>(p.q) + r * p.q_stride + ((int64_t)head * p.group + h0 + min(g, n_heads - 1)) * D, asks, t, x);
  fetch(0);
#pragma unroll 1
  for (int j = 0; j < ST; ++j) issue(j, ring + j * L::kSlot);
  W st;
  st.set_q(x, t, p.scale);
  uint32_t slot = warp * ST * L::kSlot;
#pragma unroll 1
  for (int j = 0; j * L::kStep < nt; ++j) {
    cp_async_wait<ST - 1>();
    __syncwarp();
    if (doubt || j < plain0 || j - plain0 >= plain_n) {
      uint64_t rows_seen = 0;  // a bit per row of the step
#pragma unroll
      for (int k = 0; k < L::kStep; ++k) {
        const int i = j * L::kStep + k, row = i < nt ? tile_row(v, tile_no(i)) : 0, at = row + (lane & 15);
        const bool sees = i < nt && (at < v.first || (at >= v.lo && at < v.len)) && page_of(row) >= 0;
        rows_seen |= (uint64_t)(__ballot_sync(0xffffffffu, sees) & 0xffff) << (16 * k);
      }
      st.template step<true>(smem + slot, lane, rows_seen);
    } else {
      st.template step<false>(smem + slot, lane, 0);
    }
    __syncwarp();
    issue(j + ST, smem_u32(smem) + slot);
    slot += L::kSlot;
    if (slot == (warp + 1) * ST * L::kSlot) slot = warp * ST * L::kSlot;
  }
  cp_async_wait<0>();

  // ---- the warps' sums, brought to one reference
  st.write_refs(warp_ref[warp], lane);
  __syncthreads();  // every warp is through with its ring
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int h = 2 * t + hh;
    float m = warp_ref[0][h].x;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, warp_ref[w][h].x);
    const float k = exp2_approx(warp_ref[warp][h].x - m);
    float* row = sums + (warp * kHeadBlock + h) * L::kMergeRow;
#pragma unroll
    for (int x = 0; x < W::NB; ++x) {
      const float kx = k * st.out_unit(x);
#pragma unroll
      for (int y = 0; y < 2; ++y)
        *reinterpret_cast<float2*>(row + W::out_dim(x, y, g)) =
            make_float2(st.acc[x][y][hh] * kx, st.acc[x][y][2 + hh] * kx);
    }
  }
  __syncthreads();
  UnitSums<D> o;
  constexpr int N = UnitSums<D>::N;
  const int h = tid / 16, e = (tid % 16) * N;
  o.m = warp_ref[0][h].x;
  o.l = 0.f;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) o.m = fmaxf(o.m, warp_ref[w][h].x);
#pragma unroll
  for (int i = 0; i < N; ++i) o.x[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    o.l += warp_ref[w][h].y * exp2_approx(warp_ref[w][h].x - o.m);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 y = *reinterpret_cast<const float4*>(sums + (w * kHeadBlock + h) * L::kMergeRow + e + i);
      o.x[i] += y.x, o.x[i + 1] += y.y, o.x[i + 2] += y.z, o.x[i + 3] += y.w;
    }
  }
  return o;
}

// Writes a unit's outputs: thread tid the N dimensions that it holds.
template <int D, class T>
__device__ __forceinline__ void write_unit(const KvAttnParams& p, int r, int u, UnitSums<D>& o) {
  const int head = u / p.head_blocks, h = (u % p.head_blocks) * kHeadBlock + threadIdx.x / 16;
  if (h >= p.group) return;
  if (!KV_IN_BOUNDS(p.c, r >= 0 && r < p.n && head < p.c.nkv)) return;
  const float k = over(o.l);
#pragma unroll
  for (int i = 0; i < o.N; ++i) o.x[i] *= k;
  store_out(static_cast<T*>(p.o) + r * p.o_stride + ((int64_t)head * p.group + h) * D + (threadIdx.x % 16) * o.N, o.x);
}

// Units that are all short: a CTA takes whole units in turn.
template <int D, bool Q4, class T>
__global__ void __launch_bounds__(kThreadsA, Tile<D, Q4>::kCtasPerSm)
    kv_attn_whole(const __grid_constant__ KvAttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int units = p.c.nkv * p.head_blocks;
  for (int id = blockIdx.x; id < p.n * units; id += gridDim.x) {
    const int r = id / units, u = id % units;
    bool bad = false;
    const Rows v = query_rows(p, r, &bad);
    if (bad && threadIdx.x == 0) atomicOr(p.c.status, DEC_KV_BAD_INDEX);
    if (v.seq < 0) continue;
    UnitSums<D> o = unit_sums<D, Q4, T>(p, v, r, u, 0, v.tiles, smem);
    write_unit<D, T>(p, r, u, o);
  }
}

// A CTA's share of the line and where it stands in it.  The line is all units
// in order, each as long as its tiles and `unit` more, which come first.
struct Share {
  int64_t pos, end;      // positions in the line
  int64_t before;        // the length of one unit each of the queries before r
  int64_t total, parts;  // length and shares of the whole line
  int r, u, t0, t1;      // the unit at hand
  int cut;               // a unit begins here that ends elsewhere
  int more;              // CTAs that the unit which begins here goes on for; -1: to be worked out
};

template <int D, bool Q4, class T>
__global__ void __launch_bounds__(kThreadsA, Tile<D, Q4>::kCtasPerSm) kv_attn(const __grid_constant__ KvAttnParams p) {
  using L = Tile<D, Q4>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t chunk_sum[kMaxChunks];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const KvView& c = p.c;
  pdl_trigger();

  // ---- this CTA's share of the line
  constexpr int kRound = kWarps * L::kStep, kLeast = kRound / 2;
  const int chunks = (p.n + kChunkRows - 1) / kChunkRows;
  const int units = c.nkv * p.head_blocks;
  bool bad = false, empty = false;
  __shared__ Share share;  // (not in registers: the products need them)
  Rows v{-1, 0, 0, 0, 0, 0, 0};
  auto hidden = [&](int r, const Rows& rows) {  // a query that sees no row, or is skipped
    if (p.cut_by_unit)
      for (int u = tid; u < units; u += kThreadsA)
        if (KV_IN_BOUNDS(c, r * units + u < p.ctas)) p.cut[r * units + u] = make_int4(0, 0, 0, 0);
    if (rows.seq < 0) return;
    T* out = static_cast<T*>(p.o) + r * p.o_stride;
    for (int64_t e = tid; e < (int64_t)p.nq * D; e += kThreadsA) out[e] = 0;
  };
  int unit = 0;  // what a unit counts besides its tiles
  if (p.n == 1 && units <= (int)gridDim.x) {
    // One query: its units are alike, each is cut into as many parts as there are
    // CTAs for it, of whole rounds if they are small.  (Counting and looking for
    // borders, below, would take 2.5 us of a short call.)
    v = query_rows(p, 0, &bad);
    if (bad && blockIdx.x == 0 && tid == 0) atomicOr(c.status, DEC_KV_BAD_INDEX);
    if (v.tiles == 0) {
      if (blockIdx.x == 0) hidden(0, v);
      return;
    }
    const int most = gridDim.x / units, even = (v.tiles + most - 1) / most;
    const int size = even <= 3 * kRound ? (even + kRound - 1) / kRound * kRound : even;
    const int cuts = (v.tiles + size - 1) / size;
    const int u = blockIdx.x / cuts, t0 = (blockIdx.x - u * cuts) * size;
    if (u >= units) return;
    if (tid == 0) {
      const int64_t first = (int64_t)u * v.tiles;
      share = Share{first + t0, first + min(t0 + size, v.tiles), 0, 0, 0, 0, 0, 0, 0, 0, cuts - 1};
    }
    __syncthreads();
  } else {
    int mine[4];  // tiles of a unit of queries 32 i + lane of a chunk
    auto count = [&](int chunk) {
      int64_t sum = 0;  // tiles, and the queries that have any from bit 48 up
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = chunk * kChunkRows + 32 * i + lane;
        Rows v{-1, 0, 0, 0, 0, 0, 0};
        if (r < p.n) v = query_rows(p, r, &bad);
        mine[i] = v.tiles;
        sum += v.tiles + ((int64_t)(v.tiles > 0) << 48);
        empty |= r < p.n && v.tiles == 0;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      return sum;
    };
    int64_t tiles = 0;
    int queries = 0;
    auto add = [&](int64_t sum) {
      tiles += sum & ((1ll << 48) - 1);
      queries += (int)(sum >> 48);
    };
    if (chunks == 1) {
      add(count(0));  // every warp for itself
    } else {
      for (int k = warp; k < chunks; k += kWarps) {
        const int64_t sum = count(k);
        if (lane == 0 && KV_IN_BOUNDS(c, k < kMaxChunks)) chunk_sum[k] = sum;
      }
      __syncthreads();
      for (int k = 0; k < chunks; ++k) add(chunk_sum[k]);
    }
    if (bad && blockIdx.x == 0) atomicOr(c.status, DEC_KV_BAD_INDEX);
    if (__syncthreads_or(empty)) {
      for (int r = blockIdx.x; r < p.n; r += gridDim.x) {
        const Rows rows = query_rows(p, r, &bad);
        if (rows.tiles == 0) hidden(r, rows);
      }
    }
    // What a unit counts besides its tiles: what it costs; but where all are long
    // and the shares short, a share has one unit at most and the cost is the same
    // for all.
    unit = tiles <= (int64_t)L::kShort * queries ? L::kUnit
                                                 : (int)min((int64_t)L::kUnit, tiles * units / (int64_t)gridDim.x);
    const int64_t total = (tiles + (int64_t)unit * queries) * units;
    // One share per CTA; small ones of whole rounds, so that every warp has as much.
    const int64_t rounds = (total + (int64_t)gridDim.x * kRound - 1) / ((int64_t)gridDim.x * kRound);
    const int64_t parts = rounds > 3 ? gridDim.x : (total + rounds * kRound - 1) / (max(rounds, (int64_t)1) * kRound);
    if (blockIdx.x >= parts) {
      if (!p.cut_by_unit && tid == 0) p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
      return;
    }
    // The border between two shares is moved to the nearer end of a unit that
    // is short, in itself or beside a share, and to an end of a long one that
    // is less than kLeast tiles off (shares are longer).
    const int64_t shortest = max((int64_t)L::kShort, total / parts / 16) + unit;
    int64_t before;
    int r, r_len;
    auto locate = [&](int64_t want) {  // the query with position `want` of the line
      want /= units;
      before = 0;
      r = r_len = 0;
      int k = 0;
      if (chunks > 1) {
        auto length = [&](int at) { return (chunk_sum[at] & ((1ll << 48) - 1)) + unit * (chunk_sum[at] >> 48); };
        while (k + 1 < chunks && before + length(k) <= want) before += length(k++);
        count(k);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int len = mine[i] ? mine[i] + unit : 0;
        int64_t incl = len;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, before + incl > want);
        if (past) {
          const int at = __ffs(past) - 1;
          r_len = __shfl_sync(0xffffffffu, len, at);
          before += __shfl_sync(0xffffffffu, incl, at) - r_len;
          r = k * kChunkRows + 32 * i + at;
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    };
    auto border = [&](int64_t part) {  // where share `part` begins
      int64_t pos = total * part / parts;
      if (pos < total) {
        locate(pos);
        if (r_len > 0) {
          const int in = (int)((pos - before * units) % r_len);
          if (r_len <= shortest) pos += 2 * in < r_len ? -in : r_len - in;
          else if (in < unit + kLeast) pos -= in;
          else if (in > r_len - kLeast) pos += r_len - in;
        }
      }
      return pos;
    };
    if (warp < 2) {  // one looks for each end
      const int64_t pos = border(blockIdx.x + warp);
      if (warp == 0 && pos < total && pos >= (before + r_len) * units) locate(pos);  // moved on to the next query
      if (tid == 0) {
        share.pos = pos, share.before = before, share.r = r;
        share.total = total, share.parts = parts, share.cut = 0, share.more = -1;
      }
      if (tid == 32) share.end = pos;
    }
    __syncthreads();
    if (share.pos < share.end) v = query_rows(p, share.r, &bad);
  }

  while (share.pos < share.end) {
    const int64_t rel = share.pos - share.before * units;
    const int len = v.tiles + unit;
    // (not so only if lengths change while the call runs: then leave, in bounds)
    if (v.tiles == 0 || rel < 0 || rel >= (int64_t)len * units) break;
    const int u = rel < 1ll << 31 ? (int)rel / len : (int)(rel / len), in = (int)(rel - (int64_t)u * len);
    const int t0 = max(in - unit, 0);
    const int t1 = max((int)min((int64_t)len, in + (share.end - share.pos)) - unit, t0);
    if (tid == 0) share.u = u, share.t0 = t0, share.t1 = t1;  // (read after the barriers within unit_sums)
    UnitSums<D> o = unit_sums<D, Q4, T>(p, v, share.r, u, t0, t1, smem);
    const bool begins = share.t0 == 0, ends = share.t1 == v.tiles;
    if (begins && ends) {
      write_unit<D, T>(p, share.r, share.u, o);
    } else {  // a part: slot 1 where the unit begins here, slot 0 where it began before
      const int64_t slot = (2 * (int64_t)blockIdx.x + begins) * kHeadBlock + tid / 16;
      if (KV_IN_BOUNDS(c, slot >= 0 && slot < 2 * (int64_t)p.ctas * kHeadBlock)) {
        store_out(p.rec + slot * D + (tid % 16) * o.N, o.x);
        if (tid % 16 == 0) p.ref[slot] = make_float2(o.m, o.l);
      }
    }
    if (begins && tid == 0) {
      int more = ends ? 0 : share.more;  // borders within the unit
      if (more < 0) {
        const int64_t first = share.before * units + (int64_t)share.u * (v.tiles + unit);
        auto owner = [&](int64_t x) { return ((x + 1) * share.parts - 1) / share.total; };
        more = (int)(owner(first + v.tiles + unit - kLeast) - owner(first + unit + kLeast - 1));
      }
      const bool there = KV_IN_BOUNDS(c, share.r >= 0 && share.r < p.n && share.u < units &&
                                             (!p.cut_by_unit || share.r * units + share.u < p.ctas));
      if (!there) more = 0;
      else if (p.cut_by_unit) p.cut[share.r * units + share.u] = make_int4(share.r, share.u, blockIdx.x, more);
      else if (more) p.cut[blockIdx.x] = make_int4(share.r, share.u, blockIdx.x, more);
      share.cut |= more;
    }
    const bool next = ends && share.u == units - 1;
    const int64_t now = share.before * units + (int64_t)share.u * (v.tiles + unit) + unit + share.t1;
    const int64_t past = share.before + v.tiles + unit;
    int at = share.r;
    if (next && now < share.end && at + 1 < p.n) {
      do v = query_rows(p, ++at, &bad);
      while (v.tiles == 0 && at + 1 < p.n);
    }
    __syncthreads();
    if (tid == 0) {
      share.pos = now;
      if (next) share.before = past, share.r = at;
    }
    __syncthreads();
  }
  if (!p.cut_by_unit && tid == 0 && !share.cut) p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
}

// Joins the parts of the units that are cut, in their order.  WARPS warps take
// the parts of one query head in turn; with one, a CTA joins all 8 heads of a
// unit, with 8 blockIdx.y is the head (few units, cut into many parts).
template <int D, class T, int WARPS>
__global__ void __launch_bounds__(256) kv_attn_join(const __grid_constant__ KvAttnParams p) {
  constexpr int N = D / 32;
  __shared__ float sums[WARPS][D + 1];
  pdl_wait();
  const int4 cut = p.cut[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = cut.w + 1;
  // (the bounds hold unless lengths changed while kv_attn ran)
  if (cut.w <= 0 || cut.x >= p.n || cut.y >= p.c.nkv * p.head_blocks || cut.z + cut.w >= p.ctas) return;
  const int h = WARPS == 1 ? warp : blockIdx.y, first = WARPS == 1 ? 0 : warp;
  const int head = cut.y / p.head_blocks, h0 = (cut.y % p.head_blocks) * kHeadBlock;
  if (h0 + h >= p.group) return;
  if (!KV_IN_BOUNDS(p.c, cut.x >= 0 && cut.y >= 0 && cut.z >= 0 && head < p.c.nkv)) return;
  auto slot = [&](int i) { return (2 * (int64_t)(cut.z + i) + (i == 0)) * kHeadBlock + h; };
  float m = -3e38f;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, p.ref[slot(i)].x);
  float x[N], l = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = 0.f;
  constexpr int kBatch = 8;  // parts whose loads are under way together
  bool know_m = false;
  for (int i0 = first; i0 < n; i0 += kBatch * WARPS) {
    float y[kBatch][N];
    float2 rl[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * WARPS;
      rl[b] = make_float2(-3e38f, 0.f);
#pragma unroll
      for (int k = 0; k < N; ++k) y[b][k] = 0.f;
      if (i < n) {
        rl[b] = p.ref[slot(i)];
        const float* src = p.rec + slot(i) * D + lane * N;
        if constexpr (N == 4) *reinterpret_cast<float4*>(y[b]) = *reinterpret_cast<const float4*>(src);
        else *reinterpret_cast<float2*>(y[b]) = *reinterpret_cast<const float2*>(src);
      }
    }
    if (!know_m) m = warp_max(m);
    know_m = true;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float w = i0 + b * WARPS < n ? exp2_approx(rl[b].x - m) : 0.f;
      l = fmaf(w, rl[b].y, l);
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = fmaf(w, y[b][k], x[k]);
    }
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) sums[warp][lane * N + k] = x[k];
    if (lane == 0) sums[warp][D] = l;
    __syncthreads();
    if (warp) return;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      l += sums[w][D];
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] += sums[w][lane * N + k];
    }
  }
  const float k = over(l);
  T* out = static_cast<T*>(p.o) + cut.x * p.o_stride + ((int64_t)head * p.group + h0 + h) * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 4) out[i] = x[i] * k;
    else out[i] = f32_to_bf16_bits(x[i] * k);
  }
}

constexpr int kMaxDevices = 64;

// SMs of the current device (they do not change: looked up once).
int device_sms(int* dev, int* sms) {
  static std::atomic<int> known[kMaxDevices];
  cudaError_t e = cudaGetDevice(dev);
  if (e == cudaSuccess && (*dev < 0 || *dev >= kMaxDevices)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess && (*sms = known[*dev].load(std::memory_order_relaxed)) == 0) {
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (e == cudaSuccess) known[*dev].store(*sms, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return fail_no_handle(DEC_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  return DEC_OK;
}

// CTAs of a launch: one round of what fits on the GPU.
int attn_ctas(const dec_kv_cache& c, int sms) {
  const bool q4 = c.format == DEC_KV_Q4B32;
  if (c.head_dim == 128) return sms * (q4 ? Tile<128, true>::kCtasPerSm : Tile<128, false>::kCtasPerSm);
  return sms * (q4 ? Tile<64, true>::kCtasPerSm : Tile<64, false>::kCtasPerSm);
}

struct Workspace {
  size_t rec, ref, cut, bytes;
};
Workspace workspace_of(int ctas, int head_dim) {
  Workspace w;
  w.rec = 0;
  w.ref = w.rec + (size_t)2 * ctas * kHeadBlock * head_dim * sizeof(float);
  w.cut = w.ref + (size_t)2 * ctas * kHeadBlock * sizeof(float2);
  w.bytes = w.cut + (size_t)ctas * sizeof(int4);
  return w;
}

// The longest unit, in tiles, of a cache of this shape.
int64_t longest_unit(const KvAttnParams& p) {
  const int64_t rows = (int64_t)p.c.max_pages * p.c.page_rows;
  return p.window ? std::min(rows, (int64_t)p.window + p.sinks) / kTileRows + 3 : (rows + kTileRows - 1) / kTileRows;
}

template <int D, bool Q4, class T>
cudaError_t launch_attn_kv(KvAttnParams p, int dev, int ctas, cudaStream_t s) {
  static std::atomic<bool> ready[kMaxDevices];  // the kernels' shared-memory limits have been set on the device
  if (!ready[dev].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(kv_attn<D, Q4, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Tile<D, Q4>::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv_attn_whole<D, Q4, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Tile<D, Q4>::kSmem);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  const int64_t units = (int64_t)p.n * p.c.nkv * p.head_blocks;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreadsA);
  cfg.dynamicSmemBytes = Tile<D, Q4>::kSmem;
  cfg.stream = s;
  if (longest_unit(p) <= Tile<D, Q4>::kWhole) {
    cfg.gridDim = dim3((unsigned)std::min(units, (int64_t)ctas));
    return cudaLaunchKernelEx(&cfg, kv_attn_whole<D, Q4, T>, p);
  }
  cfg.gridDim = dim3(ctas);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attn<D, Q4, T>, p);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute pdl = {};
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  if (!p.cut_by_unit) return cudaLaunchKernelEx(&cfg, kv_attn_join<D, T, 1>, p);
  if (units > ctas / kHeadBlock) {
    cfg.gridDim = dim3((unsigned)units);
    return cudaLaunchKernelEx(&cfg, kv_attn_join<D, T, 1>, p);
  }
  cfg.gridDim = dim3((unsigned)units, std::min(kHeadBlock, p.group));
  return cudaLaunchKernelEx(&cfg, kv_attn_join<D, T, 8>, p);
}

int check_attention(const dec_kv_cache* c, int n, int n_q_heads) {
  if (n < 0 || n > kMaxQueries) return fail_no_handle(DEC_ERR_ARG, "%d queries (0..%d)", n, kMaxQueries);
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || n_q_heads > 65536)
    return fail_no_handle(DEC_ERR_SHAPE, "%d query heads: a multiple of the %d KV heads", n_q_heads, c->n_kv_heads);
  if ((int64_t)n * n_q_heads > 1 << 24)
    return fail_no_handle(DEC_ERR_SHAPE, "%d queries of %d heads (at most 2^24 in all)", n, n_q_heads);
  return DEC_OK;
}

}  // namespace

extern "C" int dec_kv_attention_workspace(const dec_kv_cache* c, size_t* bytes) {
  if (int rc = kv_check(c, false)) return rc;
  if (!bytes) return fail_no_handle(DEC_ERR_ARG, "bytes is NULL");
  int dev = 0, sms = 0;
  if (int rc = device_sms(&dev, &sms)) return rc;
  *bytes = workspace_of(attn_ctas(*c, sms), c->head_dim).bytes;
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
  // (in log2 units, as the kernels take it: past fp32 it would make scores of 0 NaN)
  const float scale2 =
      (float)((scale != 0.f ? (double)scale : 1.0 / std::sqrt((double)c->head_dim)) * 1.4426950408889634);
  if (!std::isfinite(scale2)) return fail_no_handle(DEC_ERR_ARG, "the scale %g is not finite, or too large", scale);
  if (!seqs && n > c->n_seqs) return fail_no_handle(DEC_ERR_ARG, "%d queries of %d sequences", n, c->n_seqs);
  if (n == 0) return DEC_OK;
  if (!q || !o) return fail_no_handle(DEC_ERR_ARG, "q or o is NULL");
  const int64_t size = type == DEC_IO_F32 ? 4 : 2, width = (int64_t)n_q_heads * c->head_dim;
  if (q_stride < width || o_stride < width || q_stride > (int64_t)1 << 40 || o_stride > (int64_t)1 << 40)
    return fail_no_handle(DEC_ERR_ARG, "q_stride or o_stride below the row's %lld elements", (long long)width);
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15) || (q_stride * size) % 16 ||
      (o_stride * size) % 16)
    return fail_no_handle(DEC_ERR_ARG, "q, o and their rows must be 16-byte aligned");
  if (kv_rows_overlap(reinterpret_cast<uintptr_t>(q), q_stride * size, reinterpret_cast<uintptr_t>(o), o_stride * size,
                      width * size, n))
    return fail_no_handle(DEC_ERR_ARG, "o overlaps q");
  int dev = 0, sms = 0;
  if (int rc = device_sms(&dev, &sms)) return rc;
  const int ctas = attn_ctas(*c, sms);
  const Workspace ws = workspace_of(ctas, c->head_dim);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) || workspace_bytes < ws.bytes)
    return fail_no_handle(DEC_ERR_ARG, "the workspace must be 16-byte aligned and of %zu bytes", ws.bytes);

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
  p.group = n_q_heads / c->n_kv_heads;
  p.head_blocks = (p.group + kHeadBlock - 1) / kHeadBlock;
  p.scale = scale2;
  p.rec = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ws.rec);
  p.ref = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + ws.ref);
  p.cut = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + ws.cut);
  p.ctas = ctas;
  p.cut_by_unit = (int64_t)n * c->n_kv_heads * p.head_blocks <= ctas;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool q4 = c->format == DEC_KV_Q4B32, f32 = type == DEC_IO_F32;
#define TLD_ATTN(D, Q)                                       \
  e = f32 ? launch_attn_kv<D, Q, float>(p, dev, ctas, s)     \
          : launch_attn_kv<D, Q, uint16_t>(p, dev, ctas, s)
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
