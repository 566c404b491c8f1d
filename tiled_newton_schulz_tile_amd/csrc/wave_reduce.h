// Reductions over a wave of 64 lanes with DPP moves, in a fixed order and without LDS: shifts by
// 1, 2, 4 and 8 within rows of 16 lanes, then the rows' last lanes to the rows after them; lane
// 63 holds the result, which every lane gets as a scalar.  All 64 lanes take part.
#pragma once

#include <hip/hip_runtime.h>

namespace himuon {
namespace dev {

// x of the lane that the move CTRL reads from; `none` where there is no such lane (or the row is
// not in ROWS)
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned dpp(unsigned none, unsigned x) {
  return (unsigned)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float none, float x) {
  return __builtin_bit_cast(float, dpp<CTRL, ROWS>(__builtin_bit_cast(unsigned, none), __builtin_bit_cast(unsigned, x)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double none, double x) {
  const unsigned long long n = __builtin_bit_cast(unsigned long long, none), v = __builtin_bit_cast(unsigned long long, x);
  const unsigned lo = dpp<CTRL, ROWS>((unsigned)n, (unsigned)v), hi = dpp<CTRL, ROWS>((unsigned)(n >> 32), (unsigned)(v >> 32));
  return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
__device__ __forceinline__ unsigned last_lane(unsigned x) { return (unsigned)__builtin_amdgcn_readlane((int)x, 63); }
__device__ __forceinline__ float last_lane(float x) {
  return __builtin_bit_cast(float, last_lane(__builtin_bit_cast(unsigned, x)));
}
__device__ __forceinline__ double last_lane(double x) {
  const unsigned long long v = __builtin_bit_cast(unsigned long long, x);
  return __builtin_bit_cast(double, (unsigned long long)last_lane((unsigned)(v >> 32)) << 32 | last_lane((unsigned)v));
}

// each lane's and all lanes' before it
template <class T, class OP>
__device__ __forceinline__ T wave_scan(T x, T none, OP op) {
  x = op(x, dpp<0x111, 0xf>(none, x));
  x = op(x, dpp<0x112, 0xf>(none, x));
  x = op(x, dpp<0x114, 0xf>(none, x));
  x = op(x, dpp<0x118, 0xf>(none, x));
  x = op(x, dpp<0x142, 0xa>(none, x));
  x = op(x, dpp<0x143, 0xc>(none, x));
  return x;
}
template <class T, class OP>
__device__ __forceinline__ T wave_reduce(T x, T none, OP op) {
  return last_lane(wave_scan(x, none, op));
}
__device__ __forceinline__ unsigned wave_max(unsigned x) {
  return wave_reduce(x, 0u, [](unsigned a, unsigned b) { return max(a, b); });
}
__device__ __forceinline__ float wave_max(float x) {
  return wave_reduce(x, -__builtin_inff(), [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float x) {
  return wave_reduce(x, 0.f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ double wave_sum(double x) {
  return wave_reduce(x, 0.0, [](double a, double b) { return a + b; });
}

}  // namespace dev
}  // namespace himuon
