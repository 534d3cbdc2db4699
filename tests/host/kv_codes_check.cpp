// The divisions that the 4-bit rows are written without (csrc/kv_rows.cu):
// x / 7 from the rounded reciprocal, and the integer nearest to x / s from a
// reciprocal that is up to 2^-23 off, with one FMA correction each, checked
// against IEEE division and against exact arithmetic in 64 bits.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>

static float bits(uint32_t b) {
  float f;
  std::memcpy(&f, &b, 4);
  return f;
}
static int32_t as_int(float f) {
  int32_t b;
  std::memcpy(&b, &f, 4);
  return b;
}

static float seventh(float x) {
  const float y = 1.f / 7;
  const float q = x * y;
  return std::fmaf(std::fmaf(-7.f, q, x), y, q);
}

// As q4_codes, for one value; `inv` is the reciprocal it is given.
static int code(float x, float s, float inv) {
  const float magic = 12582912.f;
  if (s < 6.103515625e-5f || s >= 65504.f) x = std::fmin(std::fmax(x, -8.f * s), 7.f * s);
  const float r0 = x * inv, r = std::fmaf(std::fmaf(r0, -s, x), inv, r0);
  return (int)((r + magic) - magic);
}

int main() {
  long bad = 0;
  for (uint32_t e : {100u, 127u, 128u, 130u, 200u})  // every mantissa
    for (uint32_t m = 0; m < (1u << 23); ++m) {
      const float x = bits(e << 23 | m);
      bad += seventh(x) != x / 7;
    }
  std::mt19937_64 rng(1);
  for (long n = 0; n < 20000000; ++n) {
    // a scale of fp16 (11 bits; below 2^-14 fewer), a value of 24 or 8 bits, many on or next to a half
    const int ex = (int)(rng() % 40) - 24;
    float s = std::ldexp((float)(1024 + rng() % 1024), ex - 10);
    if (ex < -14) s = std::ldexp(std::rint(std::ldexp(s, 24)), -24);
    if (rng() % 64 == 0) s = 65504.f;
    if (s <= 0.f || s > 65504.f) continue;
    float x;
    if (rng() % 2) {
      x = (float)(((int)(rng() % 14) - 7 + 0.5) * (double)s);  // (a block's values are within 7.0035 s)
      x = bits((uint32_t)(as_int(x) + (int)(rng() % 5) - 2));
    } else {
      x = (float)(((double)(rng() >> 11) / 9007199254740992.0 * 2 - 1) * (s >= 65504.f ? 1e6 : s < 6.103515625e-5f ? 11 : 7.0033) * s);
    }
    if (rng() % 2) x = bits((uint32_t)as_int(x) & 0xffff0000u);
    if (!std::isfinite(x)) continue;
    double want = std::nearbyint((double)x / (double)s);  // (exact at halves: 24 bits over 11)
    want = std::fmin(std::fmax(want, -8.0), 7.0);
    const float inv = 1.f / s;
    for (int off = -1; off <= 1; ++off)
      if (code(x, s, bits((uint32_t)(as_int(inv) + off))) != (int)want && bad++ < 5)
        std::printf("%a / %a: %d, not %d\n", x, s, code(x, s, bits((uint32_t)(as_int(inv) + off))), (int)want);
  }
  if (bad) std::printf("%ld differ\n", bad);
  else std::printf("OK\n");
  return bad != 0;
}
