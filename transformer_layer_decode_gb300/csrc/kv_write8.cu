// Rows written into 8-bit pages: dec_kv_append and dec_kv_append_rotated of caches
// whose blocks of 16 rows of a head share a scale.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kv.h"
#include "rope.cuh"
#include "rows.cuh"

using namespace tld;

namespace {

constexpr int kThreads8 = 256;
constexpr int kTokens8 = 16;     // list entries of a CTA of write_blocks, at most
static_assert(kTokens8 * kBlockRows == kThreads8, "a thread for each row of each entry's block");
// Lists up to this length are looked through by every CTA; of longer ones a launch before
// notes who writes which row (512 rows of 8 heads: 4.8 us, noted 6.0; 1024: 6.3 and 7.4;
// 2048: 10.0 and 7.7.  Of 2 heads 4.1 and 5.7, 5.2 and 5.7, 8.1 and 6.1).
constexpr int kListed = 1024;
// CTAs of write_blocks, where the heads are enough for them (1000 rows of 32 heads of
// bf16: 912 CTAs 13.0 us, 1216 11.8, 1824 11.0; 8185 rows: 43.5, 40.2, 39.2, but 2432 41.1).
constexpr int kBlockCtas = 8 * kSms;
// With keys that turn each begins with the angles of its blocks (4093 rows of 8 heads and 32
// of queries: 24.4 us, 1216 CTAs 27.2; the other way round where a block has many heads:
// 1000 rows of 32 and 128 heads 36.9, and 25.6).
constexpr int kTurnedCtas = 3 * kSms;
constexpr uint32_t kLeastScale = 1u << 23, kMostScale = 248u << 23;  // 2^-126, 2^121

// The entry that writes each row: owners[page][row], for write_blocks' CTAs.  (What
// other calls left there is told apart by looking the entry up in the list.)
__global__ void __launch_bounds__(256) kv_owners(const __grid_constant__ KvView c, const int32_t* seqs,
                                                 const int32_t* positions, int n) {
  pdl_wait();
  pdl_trigger();
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const KvPlace at = kv_place(c, seqs, positions, t, n);
  if (at.page) c.owners[(at.page - c.pool) / c.page_bytes * c.page_rows + at.row] = (int)t;
}

// The scale of a block whose largest magnitude has the bits `top`: 2^e, the least with
// top <= 127 * 2^e.  127 is 2^7 less a 128th, so a significand of up to 127 / 64 fits
// the exponent below its own power by 6; adding 0x1ffff carries the larger ones on.
__device__ __forceinline__ uint32_t scale_for(uint32_t top) {
  if (top >= 0x7f800000u) return 0x7fffffffu;  // an infinity or NaN among them
  const uint32_t e = (top + 0x1ffffu) & 0xff800000u;
  return min(max(e, kLeastScale + (6u << 23)) - (6u << 23), kMostScale);
}
// 1 / s of a power of two of 2^-126 to 2^126.
__device__ __forceinline__ float inverse(uint32_t s) { return __uint_as_float(0x7f000000u - s); }

// The four bytes whose integers are in the low bits of m0 .. m3.
__device__ __forceinline__ uint32_t four_bytes(float m0, float m1, float m2, float m3) {
  return __byte_perm(__byte_perm(__float_as_uint(m0), __float_as_uint(m1), 0x0040),
                     __byte_perm(__float_as_uint(m2), __float_as_uint(m3), 0x0040), 0x5410);
}

// For the largest scale, which may be too small.
__device__ __forceinline__ void clamp8(float (&x)[8], uint32_t s) {
  if (s != kMostScale) return;
  const float most = 127.f * __uint_as_float(kMostScale);
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = fminf(fmaxf(x[k], -most), most);
}

// The codes of eight values for the scale s.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], uint32_t s) {
  const Two inv(inverse(s)), magic(kMagic + 128.f);
  float2 m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = fma2(Two(x[2 * k], x[2 * k + 1]), inv, magic).get();
  return make_uint2(four_bytes(m[0].x, m[0].y, m[1].x, m[1].y), four_bytes(m[2].x, m[2].y, m[3].x, m[3].y));
}

// Eight kept codes, whose scale becomes 1 / ratio of what it was.
__device__ __forceinline__ uint2 fewer8(uint2 w, float ratio) {
  auto four = [&](uint32_t u) {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaf((float)((int)(u >> (8 * k) & 255) - 128), ratio, kMagic + 128.f);
    return four_bytes(m[0], m[1], m[2], m[3]);
  };
  return make_uint2(four(w.x), four(w.y));
}

// A block's new scale from the largest magnitude written and, where rows are kept, what
// it was; a NaN stays.
__device__ __forceinline__ uint32_t new_scale(uint32_t top, uint32_t was, bool keeps) {
  const uint32_t s = scale_for(top);
  return keeps ? max(s, was == 0x7f800000u ? 0x7fffffffu : was) : s;
}

// The place of a block's scale in its page, and of its codes.
struct Block8 {
  uint8_t* codes;
  uint32_t* scale;
};
template <int D>
__device__ __forceinline__ Block8 block_at(const KvView& c, uint8_t* page, int item, int row0) {
  const int which = item >= c.nkv, head = item - which * c.nkv;
  uint8_t* half = page + which * c.half_bytes;
  return Block8{half + head * c.head_bytes + row0 * D,
                reinterpret_cast<uint32_t*>(half + c.nkv * c.head_bytes) + head * (c.page_rows / kBlockRows) +
                    row0 / kBlockRows};
}
__device__ __forceinline__ bool block_fits(const KvView& c, const uint8_t* page, int row0) {
  return KV_IN_BOUNDS(c, page >= c.pool && page + c.page_bytes <= c.pool + c.n_pages * c.page_bytes && row0 >= 0 &&
                             row0 % kBlockRows == 0 && row0 + kBlockRows <= c.page_rows &&
                             c.nkv * c.head_bytes < c.half_bytes);
}

// What both kernels are given.
template <class T>
struct Write8 {
  KvView c;
  const T *k, *v;
  int64_t stride;
  const int32_t *seqs, *positions;
  int n;
  int blocks;  // CTAs that write; those from there on rotate queries
  RopeRows q;  // and the rotation of keys
};

// A row of its own block for each list entry (a decode step): D / 8 lanes take a row of a
// head, of K or V.
template <int D, class T, bool ROPE>
__global__ void __launch_bounds__(kThreads8) write_rows(const __grid_constant__ Write8<T> p) {
  constexpr int LANES = D / 8, ITEMS = kThreads8 / LANES;
  extern __shared__ __align__(16) float q_angles[];
  __shared__ __align__(16) float angles[ROPE ? 2 : 1][ROPE ? (ITEMS / 2 + 1) * (D / 2) : 1];
  const KvView& c = p.c;
  pdl_wait();
  pdl_trigger();
  if constexpr (ROPE) {
    if ((int)blockIdx.x >= p.blocks) {
      rope_rows<T>(p.q, blockIdx.x - p.blocks, q_angles, [&](int64_t t) {
        const KvPlace at = kv_place(c, p.seqs, p.positions, t, p.n);
        return at.page ? at.pos : -1;
      });
      return;
    }
  }
  const int tid = threadIdx.x, l = tid % LANES, items = 2 * c.nkv;
  const int64_t id0 = (int64_t)blockIdx.x * ITEMS, id = id0 + tid / LANES, t = id / items;
  const int item = (int)(id - t * items);
  const bool is_key = item < c.nkv, real = t < p.n;
  Piece<T, ROPE> in{};
  const T* row = is_key ? p.k + t * p.stride + item * D : p.v + t * p.stride + (item - c.nkv) * D;
  if (real) {
    if (ROPE && is_key) in.load(row, l, p.q.r);
    else in.own.load(row + 8 * l);
  }
  const KvPlace at = kv_place(c, p.seqs, p.positions, t, p.n);
  const int r = at.row % kBlockRows, row0 = at.row - r;
  const bool ok = at.page && block_fits(c, at.page, row0);
  const Block8 b = block_at<D>(c, ok ? at.page : c.pool, item, ok ? row0 : 0);
  const uint32_t was = ok && r ? *b.scale & 0x7f800000u : 0;
  float x[8];
  if constexpr (ROPE) {
    const int half = p.q.r.rot / 2;
    const int64_t first = id0 / items;
    const int tokens = (int)min((id0 + ITEMS - 1) / items, (int64_t)p.n - 1) - (int)first + 1;
    for (int e = tid; e < tokens * half; e += kThreads8) {
      const int a = e / half, i = e - a * half;
      const KvPlace of = kv_place(c, p.seqs, p.positions, first + a, p.n);
      if (!of.page) continue;
      const float2 y = rope_angle(p.q.r, of.pos, i);
      const int at = angle_at<D>(a, i);
      angles[0][at] = y.x, angles[1][at] = y.y;
    }
    __syncthreads();
    const float* cs = angles[0] + (t - first) * (D / 2);
    if (is_key && ok) turned<D>(in, x, row, l, p.q.r, cs, cs + (angles[1] - angles[0]));
    else in.own.values(x);
  } else {
    in.own.values(x);
  }
  Eight<float> all;
  all.set(x);
  uint32_t top = __float_as_uint(all.top_here());
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (!ok) return;
  const uint32_t s = new_scale(top, was, r != 0);
  if (r && s != was && s < 0x7f800000u) {  // the kept rows, to the new steps
    const float ratio = __uint_as_float(was) * inverse(s);
#pragma unroll 5
    for (int i = 0; i < kBlockRows - 1; ++i) {
      if (i >= r) break;
      uint2* old = reinterpret_cast<uint2*>(b.codes + i * D) + l;
      *old = fewer8(*old, ratio);
    }
  }
  clamp8(x, s);
  reinterpret_cast<uint2*>(b.codes + r * D)[l] = codes8(x, s);
  if (l == 0) *b.scale = s;
}

// How a row is turned: not at all; dimensions whose partners are an aligned eight of their
// own; neighbours; dimensions whose partners lie anywhere.
enum Turn { TURN_NONE, TURN_EIGHTS, TURN_PAIRS, TURN_ODD };

// Where a lane's two eights of a row lie, of D / 16 lanes: 8 c and D / 2 + 8 c, or those
// that turn with each other.
template <int D, int TURN>
struct Eights {
  int at[2];
  bool turns;  // with each other
  __device__ __forceinline__ Eights(int c, const RopeView& r) {
    at[0] = 8 * c, at[1] = D / 2 + 8 * c, turns = false;
    const int half = r.rot / 2;
    if (TURN != TURN_EIGHTS) return;
    turns = 8 * c < half;
    at[0] = turns ? 8 * c : r.rot + 16 * (c - half / 8);
    at[1] = turns ? half + 8 * c : at[0] + 8;
  }
};

// One head's block, by a warp: rows `of` (list entries, or -1; smem), the first of them
// `first`.  D / 16 lanes have a row, 512 / D rows at a time; lanes whose row is not
// written load the first one, which leaves the largest magnitude what it is.
template <int D, class T, int TURN>
__device__ __forceinline__ void write_block(const T* x, int64_t stride, const int* of, int first,
                                            const Block8& b, const RopeView& rope, const float* cs, const float* sn) {
  constexpr int LANES = D / 16, RPR = 32 / LANES, ROUNDS = kBlockRows / RPR;
  const int lane = threadIdx.x & 31, ci = lane % LANES, r0 = lane / LANES;
  const Eights<D, TURN> e(ci, rope);
  Eight<T> in[ROUNDS][2];
  uint32_t written = 0;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int t = of[i * RPR + r0];
    written |= (uint32_t)(t >= 0) << i;
    const T* row = x + (t >= 0 ? t : of[first]) * stride;
#pragma unroll
    for (int k = 0; k < 2; ++k) in[i][k].load(row + e.at[k]);
  }
  const uint32_t was = first ? *b.scale & 0x7f800000u : 0;
  // Row i's two eights, turned.
  auto values = [&](int i, float (&y)[2][8]) {
    in[i][0].values(y[0]);
    in[i][1].values(y[1]);
    const int r = written >> i & 1 ? i * RPR + r0 : first;
    if constexpr (TURN == TURN_EIGHTS) {
      if (e.turns) {
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
          const float4 co = *reinterpret_cast<const float4*>(cs + angle_at<D>(r, 8 * ci + q));
          const float4 si = *reinterpret_cast<const float4*>(sn + angle_at<D>(r, 8 * ci + q));
          rope_turn(y[0][q], y[1][q], co.x, si.x);
          rope_turn(y[0][q + 1], y[1][q + 1], co.y, si.y);
          rope_turn(y[0][q + 2], y[1][q + 2], co.z, si.z);
          rope_turn(y[0][q + 3], y[1][q + 3], co.w, si.w);
        }
      }
    } else if constexpr (TURN == TURN_PAIRS) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
          const float4 co = *reinterpret_cast<const float4*>(cs + angle_at<D>(r, e.at[k] / 2));
          const float4 si = *reinterpret_cast<const float4*>(sn + angle_at<D>(r, e.at[k] / 2));
          if (e.at[k] < rope.rot) rope_turn(y[k][0], y[k][1], co.x, si.x);
          if (e.at[k] + 2 < rope.rot) rope_turn(y[k][2], y[k][3], co.y, si.y);
          if (e.at[k] + 4 < rope.rot) rope_turn(y[k][4], y[k][5], co.z, si.z);
          if (e.at[k] + 6 < rope.rot) rope_turn(y[k][6], y[k][7], co.w, si.w);
        }
    } else if constexpr (TURN == TURN_ODD) {
      const T* row = x + of[r] * stride;
      const int half = rope.rot / 2;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int d = e.at[k] + j;
          if (d >= rope.rot) continue;
          const int pair = d < half ? d : d - half, at = angle_at<D>(r, pair);
          const float other = value_of(row[d < half ? d + half : d - half]);
          y[k][j] = fmaf(y[k][j], cs[at], d < half ? -other * sn[at] : other * sn[at]);
        }
    }
  };
  // (Turned for the scale and again for the codes, from half the registers, took longer:
  // 4093 rows of 8 heads 17.3 us against 16.2.)
  Eight<std::conditional_t<TURN != TURN_NONE, float, T>> have[ROUNDS][2];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    float y[2][8];
    if constexpr (TURN != TURN_NONE) values(i, y);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (TURN != TURN_NONE) have[i][k].set(y[k]);
      else have[i][k] = in[i][k];
      top = largest(top, have[i][k].top_here(), 0.f);
    }
  }
  const uint32_t s = new_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(top)), was, first != 0);
  if (first && s != was && s < 0x7f800000u) {  // the kept rows, to the new steps
    const float ratio = __uint_as_float(was) * inverse(s);
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      uint4* at = reinterpret_cast<uint4*>(b.codes + (i * RPR + r0) * D) + ci;
      if (i * RPR + r0 < first) {
        const uint4 w = *at;
        const uint2 lo = fewer8(make_uint2(w.x, w.y), ratio), hi = fewer8(make_uint2(w.z, w.w), ratio);
        *at = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    float y[2][8];
    have[i][0].values(y[0]), have[i][1].values(y[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      clamp8(y[k], s);
      if (written >> i & 1) *reinterpret_cast<uint2*>(b.codes + (i * RPR + r0) * D + e.at[k]) = codes8(y[k], s);
    }
  }
  if (lane == 0) *b.scale = s;
}

// Rows of any list.  For `tokens` list entries a CTA finds the entries that write rows of
// the same blocks; the entry of a block's lowest row has the block written, its heads of
// K and V a warp each.  `splits` CTAs share the heads.
template <int D, class T, bool ROPE>
__global__ void __launch_bounds__(kThreads8, sizeof(T) == 4 ? 2 : ROPE ? 3 : 4)
    write_blocks(const __grid_constant__ Write8<T> p, int tokens, int splits, int per_split, bool listed) {
  extern __shared__ __align__(16) float q_angles[];
  __shared__ KvPlace place[kTokens8];
  __shared__ int of[kTokens8][kBlockRows];
  __shared__ int first_row[kTokens8];  // of a block that this entry has written, else -1
  __shared__ __align__(16) float angles[ROPE ? 2 : 1][ROPE ? kBlockRows * (D / 2) : 1];
  const KvView& c = p.c;
  pdl_wait();
  pdl_trigger();
  if constexpr (ROPE) {
    if ((int)blockIdx.x >= p.blocks) {
      rope_rows<T>(p.q, blockIdx.x - p.blocks, q_angles, [&](int64_t t) {
        const KvPlace at = kv_place(c, p.seqs, p.positions, t, p.n);
        return at.page ? at.pos : -1;
      });
      return;
    }
  }
  const int tid = threadIdx.x, warp = tid >> 5;
  const int chunk = blockIdx.x / splits, begin = (blockIdx.x - chunk * splits) * per_split;
  const int end = min(begin + per_split, 2 * c.nkv);
  const int64_t t0 = (int64_t)chunk * tokens;
  const int a = tid / kBlockRows, ar = tid % kBlockRows;
  bool may = false;  // have a block written: not behind an entry that writes a lower row of it
  if (tid < tokens) {
    const int64_t t = t0 + tid;
    bool second = false;
    if (t > 0 && t < p.n) {
      const int was = p.positions[t - 1], now = p.positions[t];
      second = p.seqs[t - 1] == p.seqs[t] && was < now && was >= 0 && was / kBlockRows == now / kBlockRows;
    }
    place[tid] = kv_place(c, p.seqs, p.positions, t, p.n);
    if (second) place[tid].page = nullptr;
    may = place[tid].page;
  }
  of[a][ar] = -1;
  if (!__syncthreads_or(may)) return;
  if (listed) {
    for (int e = tid; e < p.n; e += kThreads8) {
      const int s = p.seqs[e], pos = p.positions[e];
      for (int i = 0; i < tokens; ++i)
        if (place[i].page && place[i].seq == s && pos >= 0 && place[i].pos / kBlockRows == pos / kBlockRows)
          atomicMax(&of[i][pos % kBlockRows], e);
    }
    __syncthreads();
  } else if (a < tokens && place[a].page) {
    const int at = place[a].row / kBlockRows * kBlockRows + ar;
    const int e = c.owners[(place[a].page - c.pool) / c.page_bytes * c.page_rows + at];
    if (e >= 0 && e < p.n && p.seqs[e] == place[a].seq && p.positions[e] == place[a].pos / kBlockRows * kBlockRows + ar)
      of[a][ar] = e;
  }
  __syncwarp();
  const uint32_t written = __ballot_sync(0xffffffffu, of[a][ar] >= 0) >> (tid & 16) & 0xffff;
  const int lowest = __ffs(written) - 1;
  if (ar == 0) first_row[a] = a < tokens && place[a].page && written && of[a][lowest] == t0 + a ? lowest : -1;
  __syncthreads();
  for (int i = 0; i < tokens; ++i) {
    const int first = first_row[i];
    if (first < 0) continue;  // another entry has this one's block written
    const int row0 = place[i].row / kBlockRows * kBlockRows;
    if (!block_fits(c, place[i].page, row0)) continue;
    if (ROPE && begin < c.nkv) {
      __syncthreads();  // the block before has been read
      const int half = p.q.r.rot / 2, pos0 = place[i].pos / kBlockRows * kBlockRows;
      for (int e = tid; e < kBlockRows * half; e += kThreads8) {
        const int ra = e / half, j = e - ra * half;
        if (of[i][ra] < 0) continue;
        const float2 y = rope_angle(p.q.r, pos0 + ra, j);
        const int at = angle_at<D>(ra, j);
        angles[0][at] = y.x, angles[ROPE][at] = y.y;
      }
      __syncthreads();
    }
    for (int item = begin + warp; item < end; item += kThreads8 / 32) {
      const Block8 b = block_at<D>(c, place[i].page, item, row0);
      const T* from = (item < c.nkv ? p.k : p.v - c.nkv * D) + item * D;
      const RopeView& rope = p.q.r;
      if (!ROPE || item >= c.nkv)
        write_block<D, T, TURN_NONE>(from, p.stride, of[i], first, b, rope, nullptr, nullptr);
      else if (rope.pairs)
        write_block<D, T, ROPE ? TURN_PAIRS : 0>(from, p.stride, of[i], first, b, rope, angles[0], angles[ROPE]);
      else if (rope.rot % 16 == 0)
        write_block<D, T, ROPE ? TURN_EIGHTS : 0>(from, p.stride, of[i], first, b, rope, angles[0], angles[ROPE]);
      else
        write_block<D, T, ROPE ? TURN_ODD : 0>(from, p.stride, of[i], first, b, rope, angles[0], angles[ROPE]);
    }
  }
}

template <int D, class T, bool ROPE>
cudaError_t launch8(const KvView& c, const void* k, const void* v, int64_t stride, const int32_t* seqs,
                    const int32_t* positions, int n, const RopeRows* q, cudaStream_t s) {
  Write8<T> p{c, static_cast<const T*>(k), static_cast<const T*>(v), stride, seqs, positions, n, 0, RopeRows{}};
  if (q) p.q = *q;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads8);
  cfg.stream = s;
  const BehindLast behind(&cfg);
  auto grid = [&](int64_t blocks) {
    p.blocks = (int)blocks;
    cfg.gridDim = dim3((unsigned)blocks);
    if (ROPE && p.q.n) {
      cfg.gridDim.x += (unsigned)rope_cut(p.q);
      cfg.dynamicSmemBytes = rope_smem(p.q);
    }
  };
  const int items = 2 * c.nkv;
  // Without positions a sequence has one row, without a list every entry is a sequence of its own.
  if (!positions || !seqs) {
    constexpr int ITEMS = kThreads8 / (D / 8);
    grid(((int64_t)n * items + ITEMS - 1) / ITEMS);
    return cudaLaunchKernelEx(&cfg, write_rows<D, T, ROPE>, p);
  }
  const bool listed = n <= kListed;
  if (!listed) {
    cudaLaunchConfig_t first = cfg;
    first.gridDim = dim3((unsigned)((n + 255) / 256));
    cudaError_t e = cudaLaunchKernelEx(&first, kv_owners, c, seqs, positions, n);
    if (e != cudaSuccess) return e;
  }
  // (n / 128 and n / 512: 1000 rows of 8 heads 7.2 and 7.6 us for 6.6, 4093 rows 9.3 and 10.4 for
  // 8.9; 1000 of 32 heads 10.2 and 17.1 for 11.6)
  const int tokens = std::min(std::max(n / 256, 1), kTokens8);
  const int64_t chunks = (n + tokens - 1) / tokens;
  const int steps = (items + kThreads8 / 32 - 1) / (kThreads8 / 32);  // a head of K or V for each warp
  const int want = (int)std::min((int64_t)steps, std::max((int64_t)1, (ROPE ? kTurnedCtas : kBlockCtas) / chunks));
  const int per_split = (steps + want - 1) / want * (kThreads8 / 32), splits = (items + per_split - 1) / per_split;
  grid(chunks * splits);
  return cudaLaunchKernelEx(&cfg, write_blocks<D, T, ROPE>, p, tokens, splits, per_split, listed);
}

}  // namespace

cudaError_t tld::kv_write8(const KvView& c, int head_dim, bool f32, const void* k, const void* v, int64_t stride,
                           const int32_t* seqs, const int32_t* positions, int n, const RopeRows* q, cudaStream_t s) {
#define TLD_WRITE8(D, T)                                                         \
  return q ? launch8<D, T, true>(c, k, v, stride, seqs, positions, n, q, s)      \
           : launch8<D, T, false>(c, k, v, stride, seqs, positions, n, q, s)
  if (head_dim == 128) {
    if (f32) TLD_WRITE8(128, float);
    TLD_WRITE8(128, uint16_t);
  }
  if (f32) TLD_WRITE8(64, float);
  TLD_WRITE8(64, uint16_t);
#undef TLD_WRITE8
}
