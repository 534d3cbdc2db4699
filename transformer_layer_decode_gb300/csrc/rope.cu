// dec_rope_rotate and what makes a rotation: rotary positions of the rows of many
// sequences.
#include <cmath>

#include "common.cuh"
#include "kv.h"
#include "rope.cuh"

using namespace tld;

namespace tld {

int rope_check(const dec_rope* r) noexcept {
  if (!r) return fail_no_handle(DEC_ERR_ARG, "the rotation is NULL");
  if (r->head_dim < 8 || r->head_dim > 1024 || r->head_dim % 8)
    return fail_no_handle(DEC_ERR_SHAPE, "head_dim %d: a multiple of 8, 8..1024", r->head_dim);
  if (r->rot_dim < 2 || r->rot_dim > r->head_dim || r->rot_dim % 2)
    return fail_no_handle(DEC_ERR_SHAPE, "rot_dim %d: even, 2..%d", r->rot_dim, r->head_dim);
  if (r->layout != DEC_ROPE_HALF && r->layout != DEC_ROPE_PAIRS)
    return fail_no_handle(DEC_ERR_ARG, "unknown rotary layout %d", r->layout);
  if (!std::isfinite(r->magnitude)) return fail_no_handle(DEC_ERR_ARG, "the magnitude %g is not finite", r->magnitude);
  if (!r->steps || (reinterpret_cast<uintptr_t>(r->steps) & 7))
    return fail_no_handle(DEC_ERR_ARG, "the steps must be given, 8-byte aligned");
  return DEC_OK;
}

RopeView rope_view(const dec_rope& r, bool backward) {
  return RopeView{r.steps, r.rot_dim, r.layout == DEC_ROPE_PAIRS, r.magnitude, backward ? -1.f : 1.f};
}

int rope_rows_check(const dec_rope* r, const void* x, void* out, int type, int64_t x_stride, int64_t out_stride, int n,
                    int n_heads, bool backward, RopeRows* p) noexcept {
  if (!x || !out) return fail_no_handle(DEC_ERR_ARG, "rows to rotate, or their results, are NULL");
  const int64_t size = type == DEC_IO_F32 ? 4 : 2, width = (int64_t)n_heads * r->head_dim;
  if (x_stride < width || out_stride < width || x_stride > (int64_t)1 << 40 || out_stride > (int64_t)1 << 40)
    return fail_no_handle(DEC_ERR_ARG, "strides %lld and %lld of rows of %lld elements", (long long)x_stride,
                          (long long)out_stride, (long long)width);
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(out);
  if (((a | b) & 15) || (x_stride * size) % 16 || (out_stride * size) % 16)
    return fail_no_handle(DEC_ERR_ARG, "rows to rotate and their results must be 16-byte aligned");
  const bool same = a == b && (x_stride == out_stride || n == 1);
  if (!same && kv_rows_overlap(a, x_stride * size, b, out_stride * size, width * size, n))
    return fail_no_handle(DEC_ERR_ARG, "the rotated rows overlap the ones to rotate");
  *p = RopeRows{rope_view(*r, backward), x, out, x_stride, out_stride, n, n_heads, r->head_dim, 0, 0, 0, same, 0, 0, 0, 0};
  return DEC_OK;
}

}  // namespace tld

namespace {

template <class T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeRows p, const int32_t* positions) {
  extern __shared__ __align__(16) float angles[];
  pdl_wait();
  pdl_trigger();
  rope_rows<T>(p, blockIdx.x, angles, [&](int64_t t) { return positions ? positions[t] : (int)t; });
}

}  // namespace

extern "C" int dec_rope_frequencies(int rot_dim, double theta, int scaling, double factor, double context, double slow,
                                    double fast, double* frequency, float* magnitude) {
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > 1024) return fail_no_handle(DEC_ERR_SHAPE, "rot_dim %d: even, 2..1024", rot_dim);
  if (!frequency) return fail_no_handle(DEC_ERR_ARG, "frequency is NULL");
  if (scaling < DEC_ROPE_PLAIN || scaling > DEC_ROPE_YARN_INDEX) return fail_no_handle(DEC_ERR_ARG, "unknown scaling %d", scaling);
  if (!(theta > 0) || !std::isfinite(theta)) return fail_no_handle(DEC_ERR_ARG, "theta %g: positive and finite", theta);
  if (scaling != DEC_ROPE_PLAIN && (!(factor > 0) || !std::isfinite(factor)))
    return fail_no_handle(DEC_ERR_ARG, "factor %g: positive and finite", factor);
  const bool yarn = scaling == DEC_ROPE_YARN || scaling == DEC_ROPE_YARN_INDEX;
  if (yarn && !(context > 0 && std::isfinite(context) && slow >= 0 && fast > slow && std::isfinite(fast)))
    return fail_no_handle(DEC_ERR_ARG, "context %g, slow %g, fast %g: context > 0 and fast > slow >= 0", context, slow, fast);
  if (scaling == DEC_ROPE_NTK && rot_dim < 4) return fail_no_handle(DEC_ERR_SHAPE, "rot_dim %d: 4 or more to scale theta", rot_dim);
  if (scaling == DEC_ROPE_YARN_INDEX && !(theta > 1))
    return fail_no_handle(DEC_ERR_ARG, "theta %g: above 1 for pairs that turn ever more slowly", theta);
  const double base = scaling == DEC_ROPE_NTK ? theta * std::pow(factor, (double)rot_dim / (rot_dim - 2)) : theta;
  constexpr double kTurn = 6.283185307179586;
  // The pair that turns r times over the context, were there one for every number.
  auto pair_of = [&](double r) { return rot_dim * std::log(context / (kTurn * r)) / (2 * std::log(theta)); };
  double first = 0, last = 0;  // DEC_ROPE_YARN_INDEX: the last pair kept, the first one divided
  if (scaling == DEC_ROPE_YARN_INDEX) {
    first = std::fmax(std::floor(pair_of(fast)), 0.0);
    last = std::fmax(std::fmin(std::ceil(pair_of(slow)), rot_dim - 1.0), first);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == DEC_ROPE_LINEAR) w /= factor;
    if (yarn) {
      const double place = scaling == DEC_ROPE_YARN ? (context * w / kTurn - slow) / (fast - slow)
                           : last > first           ? 1 - (i - first) / (last - first)
                                                    : (i <= first ? 1.0 : 0.0);
      const double keep = std::fmin(std::fmax(place, 0.0), 1.0);
      w = w * keep + w / factor * (1 - keep);
    }
    frequency[i] = w;
  }
  if (magnitude) *magnitude = yarn ? (float)(0.1 * std::log(factor) + 1) : 1.f;
  return DEC_OK;
}

// frequency / (2 pi) in two doubles that add up to it (2 pi's inverse has two, too: the
// product is good to 2^-100), its whole turns taken off, in 2^-64.
extern "C" int dec_rope_steps(const double* frequency, int n, uint64_t* steps) {
  if (n < 0 || (n > 0 && (!frequency || !steps))) return fail_no_handle(DEC_ERR_ARG, "frequencies or steps are missing");
  constexpr double kInverse = 0x1.45f306dc9c883p-3, kRest = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
  for (int i = 0; i < n; ++i) {
    const double f = frequency[i];
    if (!(std::fabs(f) <= 1e6)) return fail_no_handle(DEC_ERR_ARG, "frequency %g: at most 1e6 radians a position", f);
    const double g = std::fabs(f), hi = g * kInverse, lo = std::fma(g, kInverse, -hi) + g * kRest;
    const double part = hi - std::floor(hi);  // (exact)
    const double top = std::floor(std::ldexp(part, 32)), rest = std::ldexp(part, 32) - top;
    const uint64_t step = ((uint64_t)top << 32) + (uint64_t)(int64_t)std::nearbyint(std::ldexp(rest, 32)) +
                          (uint64_t)(int64_t)std::nearbyint(std::ldexp(lo, 64));
    steps[i] = f < 0 ? 0 - step : step;
  }
  return DEC_OK;
}

extern "C" int dec_rope_rotate(const dec_rope* r, const void* x, void* out, int type, int64_t x_stride, int64_t out_stride,
                               const int32_t* positions, int n, int n_heads, int backward, dec_stream_t stream) {
  if (int rc = rope_check(r)) return rc;
  if (type != DEC_IO_F32 && type != DEC_IO_BF16) return fail_no_handle(DEC_ERR_ARG, "unknown type %d", type);
  if (n < 0) return fail_no_handle(DEC_ERR_ARG, "%d rows", n);
  if (n_heads < 1 || n_heads > 65536 || (int64_t)n * n_heads > (int64_t)1 << 30)
    return fail_no_handle(DEC_ERR_SHAPE, "%d rows of %d heads (1..65536, and at most 2^30 in all)", n, n_heads);
  if (n == 0) return DEC_OK;
  RopeRows p;
  if (int rc = rope_rows_check(r, x, out, type, x_stride, out_stride, n, n_heads, backward != 0, &p)) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rope_cut(p));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.dynamicSmemBytes = rope_smem(p);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  const BehindLast behind(&cfg);
  const cudaError_t e = type == DEC_IO_F32 ? cudaLaunchKernelEx(&cfg, rope_kernel<float>, p, positions)
                                           : cudaLaunchKernelEx(&cfg, rope_kernel<uint16_t>, p, positions);
  if (e != cudaSuccess) return fail_no_handle(DEC_ERR_CUDA, "rotation launch: %s", cudaGetErrorString(e));
  return DEC_OK;
}
