// Pieces of the kernels that take the softmax of rows of logits (fp32 or bf16, any element
// alignment): 16-byte vectors of a row, a thread's part of the softmax and its join over a block.
#pragma once

#include "device_common.h"
#include "wave_reduce.h"

namespace himuon {
namespace {

using namespace dev;

constexpr double kLog2e = 1.4426950408889634074;
constexpr float kLn2 = 0.69314718055994530942f;

// 16 bytes of a row, at any element alignment.
typedef unsigned u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));

template <class T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr unsigned kLowest = 0xff800000u;   // -inf in every element
  static __device__ __forceinline__ u32x4 load(const float *p) {
    return *reinterpret_cast<const GLOBAL_AS u32x4a4 *>(gmem(p));
  }
  template <bool NT>
  static __device__ __forceinline__ void store(float *p, const float (&x)[4]) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_bit_cast(unsigned, x[e]);
    GLOBAL_AS u32x4a4 *q = reinterpret_cast<GLOBAL_AS u32x4a4 *>(gmem(p));
    if constexpr (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
  }
  static __device__ __forceinline__ void unpack(u32x4 v, float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned u = v[e];
      x[e] = __builtin_bit_cast(float, u);
    }
  }
  static __device__ __forceinline__ float load1(const float *p) { return *gmem(p); }
  static __device__ __forceinline__ void store1(float *p, float x) { *gmem(p) = x; }
};
template <>
struct Vec<__bf16> {
  static constexpr int N = 8;
  static constexpr unsigned kLowest = 0xff80ff80u;
  static __device__ __forceinline__ u32x4 load(const __bf16 *p) {
    return *reinterpret_cast<const GLOBAL_AS u32x4a2 *>(gmem(reinterpret_cast<const unsigned short *>(p)));
  }
  template <bool NT>
  static __device__ __forceinline__ void store(__bf16 *p, const float (&x)[8]) {
    const u32x4 v = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    GLOBAL_AS u32x4a2 *q = reinterpret_cast<GLOBAL_AS u32x4a2 *>(gmem(reinterpret_cast<unsigned short *>(p)));
    if constexpr (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
  }
  static __device__ __forceinline__ void unpack(u32x4 v, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned u = v[e];
      x[2 * e] = __builtin_bit_cast(float, u << 16);
      x[2 * e + 1] = __builtin_bit_cast(float, u & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float load1(const __bf16 *p) {
    return bf16_bits_to_f32(*gmem(reinterpret_cast<const unsigned short *>(p)));
  }
  static __device__ __forceinline__ void store1(__bf16 *p, float x) {
    *gmem(reinterpret_cast<unsigned short *>(p)) = to_bf16_bits(x);
  }
};

// A row's softmax: ref is the largest logit (0 where there is nothing but -inf, whose powers
// are 0 then) and sum = sum_j 2^((z_j - ref) k).  The difference is taken before the product,
// so that logits near the ends of their type (a mask of its lowest value) overflow to a power
// of 0 and to nothing else.  NaN and +inf make the sum NaN.
struct Softmax {
  float ref, sum;
};
__device__ __forceinline__ float ref_of(float max) { return max == -__builtin_inff() ? 0.f : max; }
__device__ __forceinline__ float pow2(float z, float k, float ref) { return __builtin_amdgcn_exp2f((z - ref) * k); }

// 2^f for |f| <= 1/2: 1 + f q(f), q the polynomial of degree 8 that interpolates (2^f - 1) / f at the Chebyshev nodes;
// within 4e-14 of itself, and 1 exactly at f = 0.
__device__ __forceinline__ double pow2_fraction(double f) {
  double q = 0x1.b63880a30e9ffp-24;
  q = __builtin_fma(q, f, 0x1.63d136366db24p-20);
  q = __builtin_fma(q, f, 0x1.ffcb9515a8016p-17);
  q = __builtin_fma(q, f, 0x1.4308ac85aa947p-13);
  q = __builtin_fma(q, f, 0x1.5d87fe86fe88ep-10);
  q = __builtin_fma(q, f, 0x1.3b2ab7181b755p-7);
  q = __builtin_fma(q, f, 0x1.c6b08d7047e52p-5);
  q = __builtin_fma(q, f, 0x1.ebfbdff823cedp-3);
  q = __builtin_fma(q, f, 0x1.62e42fefa39efp-1);
  return __builtin_fma(q, f, 1.);
}
// 2^x for x <= 0 (0 where fp64 underflows; NaN is NaN).
__device__ __forceinline__ double pow2_exact(double x) {
  x = x < -1100. ? -1100. : x;
  const double n = __builtin_rint(x);
  return __builtin_amdgcn_ldexp(pow2_fraction(x - n), (int)n);
}

// Joins the threads' softmaxes over a block of W waves; lds holds W entries.
template <int W>
__device__ __forceinline__ Softmax block_softmax(float max, float sum, float k, Softmax *lds) {
  const int lane = threadIdx.x & 63;
  const float m = wave_max(max);
  float to = ref_of(m);
  sum = wave_sum(sum * pow2(max, k, to));   // (a thread with nothing but -inf has sum 0 and power 0)
  if constexpr (W == 1) return {to, sum};
  if (lane == 0) lds[threadIdx.x >> 6] = {m, sum};   // the maximum itself here
  __syncthreads();
  const Softmax s = lds[lane % W];
  to = ref_of(wave_max(s.ref));
  return {to, wave_sum(lane < W ? s.sum * pow2(s.ref, k, to) : 0.f)};
}

// Makes the compiler unpack a held vector anew where it is used next, rather than keep the
// unpacked floats of one pass over the row for the next (twice the registers for bf16).
__device__ __forceinline__ void hold_packed(u32x4 &v) { asm volatile("" : "+v"(v)); }

template <class T>
__device__ __forceinline__ float max_of(u32x4 v, float m) {
  float x[Vec<T>::N];
  Vec<T>::unpack(v, x);
#pragma unroll
  for (int e = 0; e < Vec<T>::N; ++e) m = __builtin_fmaxf(m, x[e]);
  return m;
}
// (by pairs: as many additions, fewer roundings of a sum that one power has already made large)
template <class T>
__device__ __forceinline__ float sum_of(u32x4 v, float k, float ref) {
  constexpr int N = Vec<T>::N;
  float x[N];
  Vec<T>::unpack(v, x);
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = pow2(x[e], k, ref);
#pragma unroll
  for (int d = 1; d < N; d *= 2)
#pragma unroll
    for (int e = 0; e < N; e += 2 * d) x[e] += x[e + d];
  return x[0];
}
template <class T, int THR, bool NT>
__device__ __forceinline__ void zero_row(T *dz, int V) {
  constexpr int N = Vec<T>::N;
  const float zero[N] = {};
  const int whole = V / N * N;
  for (int j = threadIdx.x * N; j < whole; j += THR * N) Vec<T>::template store<NT>(dz + j, zero);
  if (whole + (int)threadIdx.x < V) Vec<T>::store1(dz + whole + threadIdx.x, 0.f);
}

}  // namespace
}  // namespace himuon
