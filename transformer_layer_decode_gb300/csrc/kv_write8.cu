// Rows written into 8-bit pages: dec_kv_append and dec_kv_append_rotated of caches
// whose blocks of 16 rows of a head share a scale.
#include <algorithm>

#include "common.cuh"
#include "kv.h"
#include "rope.cuh"
#include "rows.cuh"

using namespace tld;

namespace {

constexpr int kWarps8 = 8;
constexpr int kThreads8 = kWarps8 * 32;
constexpr int kTokens8 = 16;     // list entries of a CTA, at most
static_assert(kTokens8 * kBlockRows == kThreads8, "a thread for each row of each entry's block");
constexpr int kListed = 512;     // lists up to this length are looked through by every CTA
constexpr uint32_t kLeastScale = 1u << 23, kMostScale = 248u << 23;  // 2^-126, 2^121

// How a CTA finds which list entries write rows of one block.
enum Find { FIND_ALONE, FIND_LIST, FIND_OWNERS };

// The entry that writes each row: owners[page][row], for kv_write8's CTAs.  (What
// other calls left there is told apart by looking the entry up in the list.)
__global__ void __launch_bounds__(256) kv_owners(const __grid_constant__ KvView c, const int32_t* seqs,
                                                 const int32_t* positions, int n) {
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

// A warp's block: rows `of` (list entries, or -1) of one head of K or V, the first of
// them `first`.
template <int D, class T, bool TURN>
__device__ __forceinline__ void write_block(const KvView& c, const T* x, int64_t stride, int64_t head_at, const int* of,
                                            int first, uint8_t* codes, uint32_t* scale_at, const RopeView& rope,
                                            const float* cs, const float* sn) {
  constexpr int LANES = D / 8, RPR = 32 / LANES, ROUNDS = kBlockRows / RPR;
  const int lane = threadIdx.x & 31, l = lane % LANES, r0 = lane / LANES;
  using In = std::conditional_t<TURN, float, T>;
  Eight<In> in[ROUNDS];
  uint32_t live = 0;  // rounds that have a row
  const uint32_t was = first ? *scale_at & 0x7f800000u : 0;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int t = of[i * RPR + r0];
    if (!__any_sync(0xffffffffu, t >= 0)) continue;
    live |= 1u << i;
    const T* row = x + max(t, 0) * stride + head_at;
    Eight<T> y{};
    if (t >= 0) y.load(row + 8 * l);
    if constexpr (TURN) {
      float v[8];
      y.values(v);
      const int at = (i * RPR + r0) * (D / 2);
      rope_eight<LANES>(rope, v, l, cs + at, sn + at, row, t >= 0);
      in[i].set(v);
    } else {
      in[i] = y;
    }
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i)
    if (live >> i & 1) top = largest(top, in[i].top_here(), 0.f);
  uint32_t s = scale_for(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  if (first) s = max(s, was == 0x7f800000u ? 0x7fffffffu : was);
  const Two inv(inverse(s)), magic(kMagic + 128.f);
  if (first && s != was && s < 0x7f800000u) {  // the kept rows, to the new steps
    constexpr int PER_ROW = D / 16, AT_ONCE = 32 / PER_ROW;
    const float ratio = __uint_as_float(was) * inverse(s);
#pragma unroll
    for (int i = 0; i < kBlockRows / AT_ONCE; ++i) {
      const int r = i * AT_ONCE + lane / PER_ROW;
      if (r >= first) continue;
      uint4* at = reinterpret_cast<uint4*>(codes + r * D) + lane % PER_ROW;
      const uint4 old = *at;
      auto fewer = [&](uint32_t w) {
        float m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          m[k] = fmaf((float)((int)(w >> (8 * k) & 255) - 128), ratio, kMagic + 128.f);
        return four_bytes(m[0], m[1], m[2], m[3]);
      };
      *at = make_uint4(fewer(old.x), fewer(old.y), fewer(old.z), fewer(old.w));
    }
  }
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    if (!(live >> i & 1)) continue;
    float v[8];
    in[i].values(v);
    if (s == kMostScale) {  // (which may be too small)
      const float most = 127.f * __uint_as_float(kMostScale);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fminf(fmaxf(v[k], -most), most);
    }
    float2 m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fma2(Two(v[2 * k], v[2 * k + 1]), inv, magic).get();
    const int r = i * RPR + r0;
    if (of[r] >= 0)
      reinterpret_cast<uint2*>(codes + r * D)[l] =
          make_uint2(four_bytes(m[0].x, m[0].y, m[1].x, m[1].y), four_bytes(m[2].x, m[2].y, m[3].x, m[3].y));
  }
  if (lane == 0) *scale_at = s;
}

// A CTA takes `tokens` list entries and finds, for each, the entries that write rows of
// the same block; the entry of a block's lowest row has the block written, its heads of
// K and V a warp each.  `splits` CTAs share the heads.  ROPE: keys are rotated on the
// way, in fp32, and the CTAs from `blocks` on rotate queries.
template <int D, class T, bool ROPE>
__global__ void __launch_bounds__(kThreads8) write8(const __grid_constant__ KvView c, const T* k, const T* v, int64_t stride,
                                                    const int32_t* seqs, const int32_t* positions, int n, int tokens,
                                                    int splits, Find find, int blocks, const __grid_constant__ RopeRows q) {
  extern __shared__ __align__(16) float q_angles[];
  __shared__ KvPlace place[kTokens8];
  __shared__ int of[kTokens8][kBlockRows];
  __shared__ __align__(16) float angles[ROPE ? 2 : 1][ROPE ? kBlockRows * (D / 2) : 1];
  if constexpr (ROPE) {
    if ((int)blockIdx.x >= blocks) {
      rope_rows<T>(q, blockIdx.x - blocks, q_angles, [&](int64_t t) {
        const KvPlace at = kv_place(c, seqs, positions, t, n);
        return at.page ? at.pos : -1;
      });
      return;
    }
  }
  const int tid = threadIdx.x, warp = tid >> 5, split = blockIdx.x % splits;
  const int64_t t0 = (int64_t)(blockIdx.x / splits) * tokens;
  if (tid < tokens) place[tid] = kv_place(c, seqs, positions, t0 + tid, n);
  of[tid / kBlockRows][tid % kBlockRows] = -1;
  if (find == FIND_OWNERS) pdl_wait();
  __syncthreads();
  if (find == FIND_ALONE) {
    if (tid < tokens) of[tid][place[tid].row % kBlockRows] = (int)(t0 + tid);
  } else if (find == FIND_LIST) {
    for (int e = tid; e < n; e += kThreads8) {
      const int s = seqs[e], pos = positions[e];
      for (int a = 0; a < tokens; ++a)
        if (place[a].page && place[a].seq == s && pos >= 0 && place[a].pos / kBlockRows == pos / kBlockRows)
          atomicMax(&of[a][pos % kBlockRows], e);
    }
  } else {
    const int a = tid / kBlockRows, r = tid % kBlockRows;
    if (a < tokens && place[a].page) {
      const int at = place[a].row / kBlockRows * kBlockRows + r;
      const int e = c.owners[(place[a].page - c.pool) / c.page_bytes * c.page_rows + at];
      if (e >= 0 && e < n && seqs[e] == place[a].seq && positions[e] == place[a].pos / kBlockRows * kBlockRows + r)
        of[a][r] = e;
    }
  }
  __syncthreads();
  const int items = 2 * c.nkv;
  for (int a = 0; a < tokens; ++a) {
    uint8_t* page = place[a].page;
    if (!page) continue;
    int first = 0;
    while (first < kBlockRows - 1 && of[a][first] < 0) ++first;
    if (of[a][first] != t0 + a) continue;  // another entry has this block written
    const int row0 = place[a].row / kBlockRows * kBlockRows;
    if (!KV_IN_BOUNDS(c, page >= c.pool && page + c.page_bytes <= c.pool + c.n_pages * c.page_bytes && row0 >= 0 &&
                             row0 + kBlockRows <= c.page_rows && c.nkv * c.head_bytes < c.half_bytes))
      continue;
    if constexpr (ROPE) {
      __syncthreads();  // the block before has been read
      const int half = q.r.rot / 2, pos0 = place[a].pos / kBlockRows * kBlockRows;
      for (int e = tid; e < kBlockRows * half; e += kThreads8) {
        const int r = e / half, i = e - r * half;
        if (of[a][r] < 0) continue;
        const float2 y = rope_angle(q.r, pos0 + r, i);
        angles[0][r * (D / 2) + i] = y.x, angles[1][r * (D / 2) + i] = y.y;
      }
      __syncthreads();
    }
    for (int item = split * kWarps8 + warp; item < items; item += splits * kWarps8) {
      const int which = item >= c.nkv, head = item - which * c.nkv;
      uint8_t* half = page + which * c.half_bytes;
      uint8_t* codes = half + head * c.head_bytes + row0 * D;
      uint32_t* scale_at = reinterpret_cast<uint32_t*>(half + c.nkv * c.head_bytes) + head * (c.page_rows / kBlockRows) +
                           row0 / kBlockRows;
      if (which) write_block<D, T, false>(c, v, stride, head * D, of[a], first, codes, scale_at, q.r, nullptr, nullptr);
      else write_block<D, T, ROPE>(c, k, stride, head * D, of[a], first, codes, scale_at, q.r, angles[0], angles[1]);
    }
  }
}

template <int D, class T>
cudaError_t launch8(const KvView& c, const void* k, const void* v, int64_t stride, const int32_t* seqs,
                    const int32_t* positions, int n, const RopeRows* q, cudaStream_t s) {
  // Without positions a sequence has one row, without a list every entry is a sequence of its own.
  const Find find = !positions || !seqs ? FIND_ALONE : n <= kListed ? FIND_LIST : FIND_OWNERS;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute pdl = {};
  if (find == FIND_OWNERS) {
    cfg.gridDim = dim3((unsigned)((n + 255) / 256));
    cfg.blockDim = dim3(256);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kv_owners, c, seqs, positions, n);
    if (e != cudaSuccess) return e;
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
  }
  const int tokens = std::min(std::max(n / 512, 1), kTokens8);
  const int per_block = (2 * c.nkv + kWarps8 - 1) / kWarps8;  // CTAs that give a warp each of a block's heads
  const int64_t chunks = (n + tokens - 1) / tokens;
  const int splits = (int)std::min((int64_t)per_block, std::max((int64_t)1, 2048 / chunks));
  const int blocks = (int)chunks * splits;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads8);
  RopeRows rows{};
  if (q) {
    rows = *q;
    if (rows.n) {
      cfg.gridDim.x += (unsigned)rope_cut(rows);
      cfg.dynamicSmemBytes = rope_smem(rows);
    }
  }
  return cudaLaunchKernelEx(&cfg, q ? write8<D, T, true> : write8<D, T, false>, c, static_cast<const T*>(k),
                            static_cast<const T*>(v), stride, seqs, positions, n, tokens, splits, find, blocks, rows);
}

}  // namespace

cudaError_t tld::kv_write8(const KvView& c, int head_dim, bool f32, const void* k, const void* v, int64_t stride,
                           const int32_t* seqs, const int32_t* positions, int n, const RopeRows* q, cudaStream_t s) {
  if (head_dim == 128)
    return f32 ? launch8<128, float>(c, k, v, stride, seqs, positions, n, q, s)
               : launch8<128, uint16_t>(c, k, v, stride, seqs, positions, n, q, s);
  return f32 ? launch8<64, float>(c, k, v, stride, seqs, positions, n, q, s)
             : launch8<64, uint16_t>(c, k, v, stride, seqs, positions, n, q, s);
}
