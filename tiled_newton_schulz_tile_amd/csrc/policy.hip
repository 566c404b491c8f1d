// Clipped policy loss with a KL term over sampled tokens, forward and gradient
// (himuon_policy_loss): a row softmax, a few scalars per row, and the gradient row.
//
// All sums, maxima and exponents are fp32 (the joined sums over rows fp64); the only
// rounding to fewer bits is that of the gradient to bf16 logits' own type.
#include "device_common.h"
#include "himuon_internal.h"

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
  static __device__ __forceinline__ void store(float *p, const float (&x)[4]) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_bit_cast(unsigned, x[e]);
    *reinterpret_cast<GLOBAL_AS u32x4a4 *>(gmem(p)) = v;
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
  static __device__ __forceinline__ void store(__bf16 *p, const float (&x)[8]) {
    *reinterpret_cast<GLOBAL_AS u32x4a2 *>(gmem(reinterpret_cast<unsigned short *>(p))) =
        u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
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

// Reductions over a wave with DPP moves (no LDS): rows of 16, then the rows' last lanes.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float old, float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, x),
                                                               CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float last_lane(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
__device__ __forceinline__ float wave_max(float x) {
  const float none = -__builtin_inff();
  x = __builtin_fmaxf(x, dpp<0x111, 0xf>(none, x));
  x = __builtin_fmaxf(x, dpp<0x112, 0xf>(none, x));
  x = __builtin_fmaxf(x, dpp<0x114, 0xf>(none, x));
  x = __builtin_fmaxf(x, dpp<0x118, 0xf>(none, x));
  x = __builtin_fmaxf(x, dpp<0x142, 0xa>(none, x));
  x = __builtin_fmaxf(x, dpp<0x143, 0xc>(none, x));
  return last_lane(x);
}
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp<0x111, 0xf>(0.f, x);
  x += dpp<0x112, 0xf>(0.f, x);
  x += dpp<0x114, 0xf>(0.f, x);
  x += dpp<0x118, 0xf>(0.f, x);
  x += dpp<0x142, 0xa>(0.f, x);
  x += dpp<0x143, 0xc>(0.f, x);
  return last_lane(x);
}

// Constants of a call in fp32.
struct PolicyParams {
  const int64_t *label;
  const float *weight, *advantage, *old_logp, *ref_logp;
  float *logp;
  float *part;        // workspace: per row, weight times (-min(u, c), kl, clipped)
  int64_t ld_logits, ld_dlogits;
  int32_t vocab;
  float k;            // log2(e) / temperature
  float inv_temp;     // 1 / temperature
  float low, high;    // 1 - clip_low, 1 + clip_high
  float kl_coef, grad_scale;
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

// What a row needs besides its logits; loaded before them, so that nothing waits later.
struct RowIn {
  float w, adv, old, ref_logp, zy;
  int32_t label;   // -1: the row is left out
};
template <class T>
__device__ __forceinline__ RowIn row_in(const T *z, int64_t row, const PolicyParams &p) {
  RowIn r;
  r.w = gmem(p.weight)[row];
  const int64_t y = gmem(p.label)[row];
  r.label = r.w != 0.f && y >= 0 && y < p.vocab ? (int32_t)y : -1;
  if (r.label < 0) return r;
  r.adv = gmem(p.advantage)[row];
  r.old = p.old_logp ? gmem(p.old_logp)[row] : 0.f;
  r.ref_logp = p.ref_logp ? gmem(p.ref_logp)[row] : 0.f;
  r.zy = Vec<T>::load1(z + r.label);
  return r;
}

// Writes a row's log probability and loss terms; returns its gradient's factor of
// (j == label) - p_j.  `first`: the one thread that writes.
__device__ __forceinline__ float row_terms(Softmax s, const RowIn &r, int64_t row, const PolicyParams &p, bool first) {
  const float lp = __builtin_fmaf(r.zy - s.ref, p.inv_temp, -kLn2 * __builtin_amdgcn_logf(s.sum));
  const float rho = p.old_logp ? expf(lp - r.old) : (lp == lp ? 1.f : lp);
  const float u = rho * r.adv;
  float clamped = rho;
  if (rho < p.low) clamped = p.low;
  if (rho > p.high) clamped = p.high;
  const float c = clamped * r.adv;
  const float d = p.ref_logp ? r.ref_logp - lp : 0.f;
  const float em1 = p.ref_logp ? expm1f(d) : 0.f;
  const bool clipped = u > c;
  if (first) {
    gmem(p.logp)[row] = lp;
    GLOBAL_AS float *part = gmem(p.part) + 3 * row;
    part[0] = r.w * -(clipped ? c : u);
    part[1] = r.w * (em1 - d);
    part[2] = clipped ? r.w : 0.f;
  }
  return ((clipped ? 0.f : -u) - p.kl_coef * em1) * r.w * p.grad_scale * p.inv_temp;
}
__device__ __forceinline__ void row_left_out(int64_t row, const PolicyParams &p, bool first) {
  if (!first) return;
  gmem(p.logp)[row] = 0.f;
#pragma unroll
  for (int k = 0; k < 3; ++k) gmem(p.part)[3 * row + k] = 0.f;
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
template <class T>
__device__ __forceinline__ float sum_of(u32x4 v, float k, float ref) {
  float x[Vec<T>::N];
  Vec<T>::unpack(v, x);
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < Vec<T>::N; ++e) s += pow2(x[e], k, ref);
  return s;
}
// A vector of the gradient: coef ((j == label) - p_j), f = -coef / sum.
template <class T>
__device__ __forceinline__ void gradient(T *p, u32x4 v, float k, float ref, float f, float coef, int label_at) {
  float x[Vec<T>::N];
  Vec<T>::unpack(v, x);
#pragma unroll
  for (int e = 0; e < Vec<T>::N; ++e) x[e] = f * pow2(x[e], k, ref);
  if ((unsigned)label_at < (unsigned)Vec<T>::N) {
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e)
      if (e == label_at) x[e] += coef;
  }
  Vec<T>::store(p, x);
}

template <class T, int THR>
__device__ __forceinline__ void zero_row(T *dz, int V) {
  constexpr int N = Vec<T>::N;
  const float zero[N] = {};
  const int whole = V / N * N;
  for (int j = threadIdx.x * N; j < whole; j += THR * N) Vec<T>::store(dz + j, zero);
  if (whole + (int)threadIdx.x < V) Vec<T>::store1(dz + whole + threadIdx.x, 0.f);
}

// One block per row, the row in registers: K vectors of 16 bytes a thread, and one element
// of the row's last V % N on the first threads.  The row is read once and the gradient
// written once; -inf stands in for what lies beyond the row.
template <typename T, int THR, int K, bool GRAD>
__global__ __launch_bounds__(THR) void policy_row_kernel(const T *logits, T *dlogits, PolicyParams p) {
  constexpr int N = Vec<T>::N;
  __shared__ Softmax lds[THR / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, V = p.vocab, vecs = V / N, rest = vecs * N + tid;
  const T *z = logits + row * p.ld_logits;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const RowIn r = row_in(z, row, p);
  if (r.label < 0) {
    row_left_out(row, p, tid == 0);
    if constexpr (GRAD) zero_row<T, THR>(dz, V);
    return;
  }
  u32x4 v[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    v[i] = u32x4{Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest};
    if (tid + i * THR < vecs) v[i] = Vec<T>::load(z + (tid + i * THR) * N);
  }
  const float tail = rest < V ? Vec<T>::load1(z + rest) : -__builtin_inff();
  float m = tail;
#pragma unroll
  for (int i = 0; i < K; ++i) m = max_of<T>(v[i], m);
  const float ref = ref_of(m);
  float sum = pow2(tail, p.k, ref);
#pragma unroll
  for (int i = 0; i < K; ++i) {
    hold_packed(v[i]);
    sum += sum_of<T>(v[i], p.k, ref);
    hold_packed(v[i]);
  }
  const Softmax s = block_softmax<THR / 64>(m, sum, p.k, lds);
  const float coef = row_terms(s, r, row, p, tid == 0);
  if constexpr (GRAD) {
    const float f = -coef / s.sum;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int j = (tid + i * THR) * N;
      if (tid + i * THR < vecs) gradient(dz + j, v[i], p.k, s.ref, f, coef, r.label - j);
    }
    if (rest < V) Vec<T>::store1(dz + rest, f * pow2(tail, p.k, s.ref) + (rest == r.label ? coef : 0.f));
  }
}

// Rows that do not fit in a block's registers: read twice, the second time mostly from the
// last-level cache (1024 threads a block keep the rows in flight below its 256 MB).
constexpr int kStreamThreads = 1024;
template <typename T, bool GRAD>
__global__ __launch_bounds__(kStreamThreads) void policy_stream_kernel(const T *logits, T *dlogits, PolicyParams p) {
  constexpr int N = Vec<T>::N, THR = kStreamThreads;
  __shared__ Softmax lds[THR / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, V = p.vocab, whole = V / N * N, rest = whole + tid;
  const T *z = logits + row * p.ld_logits;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const RowIn r = row_in(z, row, p);
  if (r.label < 0) {
    row_left_out(row, p, tid == 0);
    if constexpr (GRAD) zero_row<T, THR>(dz, V);
    return;
  }
  const float tail = rest < V ? Vec<T>::load1(z + rest) : -__builtin_inff();
  float m = tail, ref = ref_of(m), sum = pow2(tail, p.k, ref);
  for (int j = tid * N; j < whole; j += THR * N) {
    const u32x4 v = Vec<T>::load(z + j);
    m = max_of<T>(v, m);
    const float to = ref_of(m);
    sum = (sum > 0.f ? sum * pow2(ref, p.k, to) : sum) + sum_of<T>(v, p.k, to);
    ref = to;
  }
  const Softmax s = block_softmax<THR / 64>(m, sum, p.k, lds);
  const float coef = row_terms(s, r, row, p, tid == 0);
  if constexpr (GRAD) {
    const float f = -coef / s.sum;
    for (int j = tid * N; j < whole; j += THR * N)
      gradient(dz + j, Vec<T>::load(z + j), p.k, s.ref, f, coef, r.label - j);
    if (rest < V) Vec<T>::store1(dz + rest, f * pow2(tail, p.k, s.ref) + (rest == r.label ? coef : 0.f));
  }
}

// stats from the rows' terms, in fp64 and a fixed order.
__global__ __launch_bounds__(1024) void policy_join_kernel(const float *part, int64_t rows, float kl_coef,
                                                           float *stats) {
  __shared__ double lds[16][3];
  double s[3] = {0, 0, 0};
  for (int64_t i = threadIdx.x; i < rows; i += 1024)
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += (double)gmem(part)[3 * i + k];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int d = 32; d; d >>= 1) s[k] += __shfl_xor(s[k], d);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6][k] = s[k];
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  double t[3] = {0, 0, 0};
  for (int i = 0; i < 16; ++i)
    for (int k = 0; k < 3; ++k) t[k] += lds[i][k];
  gmem(stats)[0] = (float)(t[0] + (double)kl_coef * t[1]);
  for (int k = 0; k < 3; ++k) gmem(stats)[1 + k] = (float)t[k];
}

template <typename T, int THR, int K>
void launch_rows(const T *z, T *dz, unsigned rows, const PolicyParams &p, hipStream_t stream) {
  if (dz)
    hipLaunchKernelGGL((policy_row_kernel<T, THR, K, true>), dim3(rows), dim3(THR), 0, stream, z, dz, p);
  else
    hipLaunchKernelGGL((policy_row_kernel<T, THR, K, false>), dim3(rows), dim3(THR), 0, stream, z, nullptr, p);
}

template <typename T>
hipError_t launch_policy_t(const himuon_policy &c, const PolicyParams &p, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  T *dz = reinterpret_cast<T *>(c.dlogits);
  const int64_t vecs = c.vocab / Vec<T>::N;
  // (a grid's x extent holds 2^31 - 1 blocks; rows beyond go into further launches)
  constexpr int64_t kRows = (int64_t)1 << 30;
  for (int64_t r = 0; r < c.rows; r += kRows) {
    const unsigned rows = (unsigned)(c.rows - r < kRows ? c.rows - r : kRows);
    PolicyParams q = p;
    q.label += r;
    q.weight += r;
    q.advantage += r;
    if (q.old_logp) q.old_logp += r;
    if (q.ref_logp) q.ref_logp += r;
    q.logp += r;
    q.part += 3 * r;
    const T *zr = z + r * c.ld_logits;
    T *dr = dz ? dz + r * c.ld_dlogits : nullptr;
    if (vecs <= 64 * 4) launch_rows<T, 64, 4>(zr, dr, rows, q, stream);
    else if (vecs <= 256 * 4) launch_rows<T, 256, 4>(zr, dr, rows, q, stream);
    else if (vecs <= 512 * 4) launch_rows<T, 512, 4>(zr, dr, rows, q, stream);
    else if (vecs <= 512 * 8) launch_rows<T, 512, 8>(zr, dr, rows, q, stream);
    else if (vecs <= 1024 * 8) launch_rows<T, 1024, 8>(zr, dr, rows, q, stream);
    else if (vecs <= 1024 * 16) launch_rows<T, 1024, 16>(zr, dr, rows, q, stream);
    else if (dr)
      hipLaunchKernelGGL((policy_stream_kernel<T, true>), dim3(rows), dim3(kStreamThreads), 0, stream, zr, dr, q);
    else
      hipLaunchKernelGGL((policy_stream_kernel<T, false>), dim3(rows), dim3(kStreamThreads), 0, stream, zr, nullptr, q);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(policy_join_kernel, dim3(1), dim3(1024), 0, stream, p.part, c.rows, p.kl_coef, c.stats);
  return hipGetLastError();
}

}  // namespace

size_t policy_workspace(const himuon_policy &p) { return ((size_t)p.rows * 3 * sizeof(float) + 7) / 8 * 8; }

hipError_t launch_policy(const himuon_policy &c, void *workspace, hipStream_t stream) {
  PolicyParams p{};
  p.label = c.label;
  p.weight = c.weight;
  p.advantage = c.advantage;
  p.old_logp = c.old_logp;
  p.ref_logp = c.ref_logp;
  p.logp = c.logp;
  p.part = reinterpret_cast<float *>(workspace);
  p.ld_logits = c.ld_logits;
  p.ld_dlogits = c.ld_dlogits;
  p.vocab = (int32_t)c.vocab;
  p.k = (float)(kLog2e / c.temperature);
  p.inv_temp = (float)(1.0 / c.temperature);
  p.low = (float)(1.0 - c.clip_low);
  p.high = (float)(1.0 + c.clip_high);
  p.kl_coef = (float)c.kl_coef;
  p.grad_scale = (float)c.grad_scale;
  return c.dtype == HIMUON_BF16 ? launch_policy_t<__bf16>(c, p, stream) : launch_policy_t<float>(c, p, stream);
}

}  // namespace himuon
