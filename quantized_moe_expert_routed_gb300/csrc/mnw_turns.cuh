// mnw_turns.cuh -- sine and cosine of position * frequency, rounded to FP32 as
// the exact values would be (but for about one in ten thousand, which are one
// step off).
//
// The angle is taken in turns and in fixed point (64-bit fraction, see
// mnw_kv_append.cu).  Its nearest 128th A of a turn comes from a table, whose
// entries are sums of two FP32 numbers; for the rest x, at most pi / 128,
//   sin(A + x) = sin A + cos A x - sin A x^2 / 2 - cos A x^3 / 6 + ...
//   cos(A + x) = cos A - sin A x - cos A x^2 / 2 + sin A x^3 / 6 + ...
// sin A + cos A x is kept to twice FP32's length; the terms from x^2 on, below
// 3e-4, are plain FP32, so the sum is within 2^-35 before its one rounding.
#pragma once
#include <cstdint>

namespace mnw {
namespace turns {

struct alignas(16) Entry {
  float s, s_low, c, c_low;  // sin A and cos A, each the sum of two
};
struct Table {
  Entry e[128];
};
constexpr double series(double x, int first) {  // x^first / first! - x^(first + 2) / (first + 2)! + ...
  double term = first ? x : 1.0, sum = 0.0;
  for (int k = first; k < 30; k += 2) {
    sum += term;
    term *= -x * x / ((k + 1) * (k + 2));
  }
  return sum;
}
constexpr Table make_table() {
  constexpr double kStep = 6.283185307179586476925 / 128;
  Table t{};
  for (int i = 0; i < 128; ++i) {
    // from the first eighth of a turn, where the series are short
    const int quarter = ((i + 16) & 127) / 32;
    const double x = kStep * (i - 32 * quarter - (i >= 112 ? 128 : 0));
    const double sx = series(x, 1), cx = series(x, 0);
    const double s = quarter == 0 ? sx : quarter == 1 ? cx : quarter == 2 ? -sx : -cx;
    const double c = quarter == 0 ? cx : quarter == 1 ? -sx : quarter == 2 ? -cx : sx;
    t.e[i].s = static_cast<float>(s);
    t.e[i].s_low = static_cast<float>(s - static_cast<double>(t.e[i].s));
    t.e[i].c = static_cast<float>(c);
    t.e[i].c_low = static_cast<float>(c - static_cast<double>(t.e[i].c));
  }
  return t;
}
__device__ const Table kTable = make_table();

// a + b x and what its rounding lost, with x = xh + xl, a = a + a_low, b = b + b_low.
__device__ __forceinline__ float with_low(float a, float a_low, float b, float b_low, float xh, float xl, float& low) {
  const float p = __fmul_rn(b, xh), pe = fmaf(b, xh, -p);
  const float s = __fadd_rn(a, p), r = __fsub_rn(s, a);
  const float se = __fadd_rn(__fsub_rn(a, __fsub_rn(s, r)), __fsub_rn(p, r));
  low = se + (pe + (a_low + fmaf(b, xl, b_low * xh)));
  return s;
}
// Of the angle with the given 64-bit fraction of a turn.
__device__ __forceinline__ void sincos_turns(uint64_t fraction, float* sn, float* co) {
  const uint64_t index = (fraction + (1ull << 56)) >> 57;
  const int64_t rest = static_cast<int64_t>(fraction - (index << 57));  // within 2^56
  // x = 2 pi 2^-64 rest, from its upper 24 bits and the 24 below them
  constexpr double kScale = 6.283185307179586476925 / 2147483648.0;  // 2^-31 turns
  constexpr float kHi = static_cast<float>(kScale), kLo = static_cast<float>(kScale - static_cast<double>(kHi));
  const float rh = static_cast<float>(static_cast<int>(rest >> 33));
  const float rl = static_cast<float>(static_cast<uint32_t>(rest >> 9) & 0xFFFFFFu) * 0x1p-24f;
  const float xh = __fmul_rn(rh, kHi), xl = fmaf(rh, kHi, -xh) + fmaf(rh, kLo, rl * kHi);
  const Entry e = kTable.e[index & 127];
  const float x2 = xh * xh;
  const float a2 = x2 * fmaf(x2, 1.f / 24.f, -0.5f);             // cos x - 1
  const float a3 = xh * x2 * fmaf(x2, 1.f / 120.f, -1.f / 6.f);  // sin x - x
  float low;
  const float s = with_low(e.s, e.s_low, e.c, e.c_low, xh, xl, low);
  *sn = s + (low + fmaf(e.s, a2, e.c * a3 - e.s * (xh * xl)));
  const float c = with_low(e.c, e.c_low, -e.s, -e.s_low, xh, xl, low);
  *co = c + (low + fmaf(e.c, a2, -e.s * a3 - e.c * (xh * xl)));
}

}  // namespace turns
}  // namespace mnw
