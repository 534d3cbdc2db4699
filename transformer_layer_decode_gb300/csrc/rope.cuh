// Rotary positions: the angles of a row and its rotation, for the kernels that
// rotate rows and those that write rotated keys into a paged cache.
#pragma once
#include <stdint.h>

#include "../../include/dec.h"
#include "rows.cuh"

namespace tld {

// A rotation, as a kernel argument.
struct RopeView {
  const uint64_t* steps;  // [rot / 2], turns per position in 2^-64
  int rot;                // dimensions turned
  int pairs;              // pairs (2 i, 2 i + 1), else (i, i + rot / 2)
  float magnitude;
  float sign;             // of the sine: -1 backward
};

// cos and sin of pair i at a position, times the magnitude.  position * step modulo
// 2^64 is the angle in turns, exactly; its upper half is a signed number of half turns
// in [-1, 1), which sincospi takes without a reduction.  What its rounding to fp32
// leaves, an angle e of 2^-25 of half a turn at most, comes on by cos(x + e) = cos x - e
// sin x and sin(x + e) = sin x + e cos x (to e^2 / 2 < 2^-47): without it the results
// of rotations are 1.6 times as far off.
__device__ __forceinline__ float2 rope_angle(const RopeView& r, int position, int i) {
  const int turn = (int)((uint64_t)(uint32_t)position * r.steps[i] >> 32);
  const float x = (float)turn;
  const float e = (float)(turn - __float2int_rz(x)) * 1.4629180792671596e-9f * r.magnitude;  // (2 pi / 2^32)
  float s, c;
  sincospif(x * 4.656612873077393e-10f, &s, &c);
  return make_float2(fmaf(c, r.magnitude, -s * e), fmaf(s, r.magnitude, c * e) * r.sign);
}

// (a, b) turned.
__device__ __forceinline__ void rope_turn(float& a, float& b, float c, float s) {
  const float x = a;
  a = fmaf(x, c, -b * s);
  b = fmaf(b, c, x * s);
}

// Rows to be rotated, [n][heads][d] of T.  A CTA takes `tokens` rows and, of these,
// `heads_per` heads.
struct RopeRows {
  RopeView r;
  const void* x;
  void* out;
  int64_t x_stride, out_stride;
  int n, heads, d;
  int tokens, heads_per, splits;  // splits: CTAs that share the heads of its rows
  int in_place;                   // the dimensions that stay need not be copied
  int turned, per_head;           // lanes of a row that turn pairs; all of them
  uint32_t by_heads, by_lanes;    // rope_over's for heads_per and per_head
};

// e / d for d given as rope_by(d), exact while e * d < 2^32.
inline uint32_t rope_by(int d) { return d == 1 ? 0 : (uint32_t)(((1ull << 32) + d - 1) / d); }
__device__ __forceinline__ int rope_over(int e, uint32_t by) { return by ? (int)__umulhi((uint32_t)e, by) : e; }

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 32;           // of a CTA, at most
constexpr int kRopeSmem = 32 * 1024;      // its cosines and sines, at most
// CTAs that the GPU holds at once (three and six an SM: 8185 rows of 32 heads 27 us each, four 25).
constexpr int kRopeCtas = 4 * kSms;

constexpr int max_int(int a, int b) { return a > b ? a : b; }

// How a launch cuts the rows; the CTAs that it takes.  Few rows: a lane's item each,
// heads dealt out where there are many.  Many: as many rows a CTA as it takes to
// have all CTAs on the GPU at once, since a CTA begins with a chain of loads and its
// angles, and only then streams.  (Queries beside rows that are written are cut the same way.)
inline int rope_cut(RopeRows& p) {
  const int items = max_int(1, p.heads * p.d / 16);  // (about: of 16 values)
  const int most = max_int(1, kRopeSmem / (p.r.rot * 4) < kRopeTokens ? kRopeSmem / (p.r.rot * 4) : kRopeTokens);
  p.tokens = max_int(kRopeThreads / items, (p.n + kRopeCtas - 1) / kRopeCtas);
  p.tokens = p.tokens < 1 ? 1 : p.tokens > most ? most : p.tokens;
  // (of many rows, too, no more heads than rope_over counts)
  p.splits = p.n < kRopeCtas / 2 ? (items + 2 * kRopeThreads - 1) / (2 * kRopeThreads) : (items + 4095) / 4096;
  p.heads_per = (p.heads + p.splits - 1) / p.splits;
  p.splits = (p.heads + p.heads_per - 1) / p.heads_per;
  // a lane has eight values and their partners, or the next eight; or else a pair, or a value
  const int half = p.r.rot / 2, stay = p.in_place ? 0 : p.d - p.r.rot;
  if (p.r.pairs) {
    p.turned = (p.r.rot + 7) / 8;
    p.per_head = p.in_place ? p.turned : p.d / 8;
  } else {
    p.turned = half % 8 ? half : half / 8;
    p.per_head = p.turned + (half % 8 ? stay : stay / 8);
  }
  p.by_heads = rope_by(p.heads_per);
  p.by_lanes = rope_by(p.per_head);
  return (p.n + p.tokens - 1) / p.tokens * p.splits;
}
inline size_t rope_smem(const RopeRows& p) { return (size_t)p.tokens * p.r.rot * sizeof(float); }

// Block `block` of rope_cut's.  position(t): of row t, negative to skip it.  smem:
// rope_smem bytes.
template <class T, class Position>
__device__ __forceinline__ void rope_rows(const RopeRows& p, int block, float* smem, Position position) {
  __shared__ int at[kRopeTokens];
  const int tid = threadIdx.x, half = p.r.rot / 2;
  const int64_t t0 = (int64_t)(p.splits > 1 ? block / p.splits : block) * p.tokens;
  const int h0 = p.splits > 1 ? block % p.splits * p.heads_per : 0, heads = min(p.heads_per, p.heads - h0);
  const T* x = static_cast<const T*>(p.x) + h0 * (int64_t)p.d;
  T* out = static_cast<T*>(p.out) + h0 * (int64_t)p.d;
  const int total = p.tokens * heads * p.per_head;
  const bool eights = p.r.pairs || half % 8 == 0;
  struct Lane {
    int t, h, c;
    Eight<T> a, b;
  };
  // (rows that are skipped are read for nothing: their positions are not known yet)
  auto fetch = [&](int e) {
    Lane y{};
    if (e >= total) return y;
    const int row = rope_over(e, p.by_lanes);
    y.c = e - row * p.per_head;
    y.t = heads == p.heads_per ? rope_over(row, p.by_heads) : row / heads;
    y.h = row - y.t * heads;
    if (t0 + y.t < p.n) {
      const T* from = x + (t0 + y.t) * p.x_stride + y.h * p.d;
      if (p.r.pairs || y.c < p.turned) y.a.load(from + 8 * y.c);
      else y.a.load(from + p.r.rot + 8 * (y.c - p.turned));
      if (!p.r.pairs && y.c < p.turned) y.b.load(from + half + 8 * y.c);
    }
    return y;
  };
  Lane now{};
  if (eights) now = fetch(tid);  // under way while the angles are worked out
  if (tid < p.tokens) at[tid] = t0 + tid < p.n ? position(t0 + tid) : -1;
  __syncthreads();
  float* sines = smem + p.tokens * half;
  for (int e = tid; e < p.tokens * half; e += kRopeThreads) {
    const int t = p.tokens > 1 ? e / half : 0;
    if (at[t] < 0) continue;
    const float2 y = rope_angle(p.r, at[t], e - t * half);
    smem[e] = y.x, sines[e] = y.y;
  }
  __syncthreads();
  const bool wide = ((reinterpret_cast<uintptr_t>(out) | p.out_stride * sizeof(T)) & 31) == 0;
  if (eights) {
    for (int e = tid; e < total; e += kRopeThreads) {
      const Lane next = fetch(e + kRopeThreads);
      if (at[now.t] >= 0) {
        T* to = out + (t0 + now.t) * p.out_stride + now.h * p.d;
        const float *cs = smem + now.t * half, *sn = sines + now.t * half;
        const int c = now.c;
        float a[8];
        now.a.values(a);
        if (p.r.pairs) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * c + i < half) rope_turn(a[2 * i], a[2 * i + 1], cs[4 * c + i], sn[4 * c + i]);
          store8(to + 8 * c, a, wide);
        } else if (c < p.turned) {
          float b[8];
          now.b.values(b);
#pragma unroll
          for (int i = 0; i < 8; ++i) rope_turn(a[i], b[i], cs[8 * c + i], sn[8 * c + i]);
          store8(to + 8 * c, a, wide);
          store8(to + half + 8 * c, b, wide);
        } else {
          store8(to + p.r.rot + 8 * (c - p.turned), a, wide);
        }
      }
      now = next;
    }
  } else {  // partners that lie in no eight of their own
    for (int e = tid; e < total; e += kRopeThreads) {
      const int row = e / p.per_head, i = e - row * p.per_head, t = row / heads, h = row - t * heads;
      if (at[t] < 0) continue;
      const T* from = x + (t0 + t) * p.x_stride + h * p.d;
      T* to = out + (t0 + t) * p.out_stride + h * p.d;
      if (i < half) {
        float a = value_of(from[i]), b = value_of(from[i + half]);
        rope_turn(a, b, smem[t * half + i], sines[t * half + i]);
        put(to[i], a), put(to[i + half], b);
      } else {
        to[i + half] = from[i + half];
      }
    }
  }
}

// Where pair i's cosine (or sine) of row r lies in a table of D / 2 of each, so that lanes
// which have eight pairs each read whole lines: the first four of each eight, then the
// second four.
template <int D>
__device__ __forceinline__ int angle_at(int r, int i) {
  return r * (D / 2) + ((i >> 2 & 1) * (D / 16) + (i >> 3)) * 4 + (i & 3);
}

// Eight values of a row, at dimension 8 l of a head: as loaded, with (TURN) those that
// they are turned with, if these are an aligned eight too.
template <class T, bool TURN>
struct Piece {
  Eight<T> own, partner;
  __device__ __forceinline__ void load(const T* row, int l, const RopeView& r) {
    own.load(row + 8 * l);
    if constexpr (TURN) {
      const int half = r.rot / 2;
      if (!r.pairs && half % 8 == 0 && 8 * l < r.rot) partner.load(row + (8 * l < half ? 8 * l + half : 8 * l - half));
    }
  }
};

// A piece's fp32 values, turned by its row's angles.
template <int D, class T>
__device__ __forceinline__ void turned(const Piece<T, true>& p, float (&x)[8], const T* row, int l, const RopeView& r,
                                       const float* cs, const float* sn) {
  const int half = r.rot / 2;
  p.own.values(x);
  if (r.pairs) {
    const float4 c = *reinterpret_cast<const float4*>(cs + angle_at<D>(0, 4 * l));
    const float4 s = *reinterpret_cast<const float4*>(sn + angle_at<D>(0, 4 * l));
    if (4 * l < half) rope_turn(x[0], x[1], c.x, s.x);
    if (4 * l + 1 < half) rope_turn(x[2], x[3], c.y, s.y);
    if (4 * l + 2 < half) rope_turn(x[4], x[5], c.z, s.z);
    if (4 * l + 3 < half) rope_turn(x[6], x[7], c.w, s.w);
  } else if (half % 8 == 0) {
    if (8 * l >= r.rot) return;
    const float sign = 8 * l < half ? -1.f : 1.f;
    const int first = 8 * l < half ? 8 * l : 8 * l - half;
    float y[8];
    p.partner.values(y);
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      const float4 c = *reinterpret_cast<const float4*>(cs + angle_at<D>(0, first + q));
      const float4 s = *reinterpret_cast<const float4*>(sn + angle_at<D>(0, first + q));
      x[q] = fmaf(x[q], c.x, sign * (y[q] * s.x));
      x[q + 1] = fmaf(x[q + 1], c.y, sign * (y[q + 1] * s.y));
      x[q + 2] = fmaf(x[q + 2], c.z, sign * (y[q + 2] * s.z));
      x[q + 3] = fmaf(x[q + 3], c.w, sign * (y[q + 3] * s.w));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 8 * l + i;
      if (e >= r.rot) continue;
      const int at = angle_at<D>(0, e < half ? e : e - half);
      const float other = value_of(row[e < half ? e + half : e - half]);
      x[i] = fmaf(x[i], cs[at], e < half ? -other * sn[at] : other * sn[at]);
    }
  }
}

// Checks a rotation; DEC_OK or the error, recorded.
int rope_check(const dec_rope* r) noexcept;
RopeView rope_view(const dec_rope& r, bool backward);
// Checks rows to be rotated and fills in *p.
int rope_rows_check(const dec_rope* r, const void* x, void* out, int type, int64_t x_stride, int64_t out_stride, int n,
                    int n_heads, bool backward, RopeRows* p) noexcept;

}  // namespace tld
