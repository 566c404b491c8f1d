// Clipped policy loss with a KL term over sampled tokens, forward and gradient
// (himuon_policy_loss): a row softmax, a few scalars per row, and the gradient row.
//
// With x_j = (z_j - max z) / ln 2 the kernel sums 2^x_j and rescales the running sum when
// the running maximum moves, so that a row is read once for its statistics.  All sums,
// maxima and exponents are fp32 (the joined sums over rows fp64); the only rounding to
// fewer bits is that of the gradient to bf16 logits' own type.
#include "device_common.h"
#include "himuon_internal.h"

namespace himuon {
namespace {

using namespace dev;

constexpr int THREADS = 512;
constexpr float kLog2e = 1.44269504088896340736f;

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned short u16x8u __attribute__((ext_vector_type(8), aligned(2)));

// 16 bytes of a row: VEC elements, at any element alignment.
template <class T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const float *p, float (&x)[4]) {
    const f32x4u v = *reinterpret_cast<const GLOBAL_AS f32x4u *>(gmem(p));
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = v[e];
  }
  static __device__ __forceinline__ void store(float *p, const float (&x)[4]) {
    *reinterpret_cast<GLOBAL_AS f32x4u *>(gmem(p)) = f32x4u{x[0], x[1], x[2], x[3]};
  }
  static __device__ __forceinline__ float load1(const float *p) { return *gmem(p); }
  static __device__ __forceinline__ void store1(float *p, float x) { *gmem(p) = x; }
};
template <>
struct Vec<__bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const __bf16 *p, float (&x)[8]) {
    const u16x8u v = *reinterpret_cast<const GLOBAL_AS u16x8u *>(gmem(p));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = bf16_bits_to_f32(v[e]);
  }
  static __device__ __forceinline__ void store(__bf16 *p, const float (&x)[8]) {
    u16x8u v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_bf16_bits(x[e]);
    *reinterpret_cast<GLOBAL_AS u16x8u *>(gmem(p)) = v;
  }
  static __device__ __forceinline__ float load1(const __bf16 *p) {
    return bf16_bits_to_f32(*gmem(reinterpret_cast<const unsigned short *>(p)));
  }
  static __device__ __forceinline__ void store1(__bf16 *p, float x) {
    *gmem(reinterpret_cast<unsigned short *>(p)) = to_bf16_bits(x);
  }
};

// Constants of a call in fp32.
struct PolicyParams {
  const int64_t *label;
  const float *weight, *advantage, *old_logp, *ref_logp;
  float *logp;
  float *part;        // workspace: per row, weight times (-min(u, c), kl, clipped)
  int64_t ld_logits, ld_dlogits;
  int32_t vocab;
  float inv_temp;     // 1 / temperature
  float low, high;    // 1 - clip_low, 1 + clip_high
  float kl_coef, grad_scale;
};

// A running softmax: the largest logit so far and the sum of exp2((z - max) k).
struct Softmax {
  float max, sum;
};
// (-inf - -inf would be NaN: what has seen nothing but -inf adds nothing)
__device__ __forceinline__ float rescale(float max, float to, float k) {
  return max == to ? 1.f : __builtin_amdgcn_exp2f((max - to) * k);
}
__device__ __forceinline__ Softmax join(Softmax a, Softmax b, float k) {
  const float m = __builtin_fmaxf(a.max, b.max);
  return {m, a.sum * rescale(a.max, m, k) + b.sum * rescale(b.max, m, k)};
}

struct RowOut {
  float max, inv_sum, coef;
};

// What a row's statistics give: its log probability, loss terms and gradient factor.
__device__ __forceinline__ RowOut row_terms(Softmax s, float zy, float w, int64_t row, const PolicyParams &p) {
  const float lp = (zy - s.max) * p.inv_temp - logf(s.sum);
  const float adv = gmem(p.advantage)[row];
  const float rho = p.old_logp ? expf(lp - gmem(p.old_logp)[row]) : (lp == lp ? 1.f : lp);
  const float u = rho * adv;
  float clamped = rho;
  if (rho < p.low) clamped = p.low;
  if (rho > p.high) clamped = p.high;
  const float c = clamped * adv;
  const float d = p.ref_logp ? gmem(p.ref_logp)[row] - lp : 0.f;
  const float em1 = expm1f(d);
  const bool clipped = u > c;
  gmem(p.logp)[row] = lp;
  GLOBAL_AS float *part = gmem(p.part) + 3 * row;
  part[0] = w * -(clipped ? c : u);
  part[1] = w * (em1 - d);
  part[2] = clipped ? w : 0.f;
  const float dlp = (clipped ? 0.f : -u) - p.kl_coef * em1;
  return {s.max, 1.f / s.sum, dlp * w * p.grad_scale * p.inv_temp};
}

template <typename T, bool GRAD>
__global__ __launch_bounds__(THREADS) void policy_row_kernel(const T *logits, T *dlogits, PolicyParams p) {
  constexpr int N = Vec<T>::N, WAVES = THREADS / 64;
  __shared__ Softmax lds[WAVES];
  __shared__ RowOut out;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, V = p.vocab;
  const T *z = logits + row * p.ld_logits;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const float w = gmem(p.weight)[row];
  const int64_t label = gmem(p.label)[row];
  const int whole = V / N * N;
  if (w == 0.f || label < 0 || label >= V) {
    if (tid == 0) {
      gmem(p.logp)[row] = 0.f;
#pragma unroll
      for (int k = 0; k < 3; ++k) gmem(p.part)[3 * row + k] = 0.f;
    }
    if constexpr (GRAD) {
      const float zero[N] = {};
      for (int j = tid * N; j < whole; j += THREADS * N) Vec<T>::store(dz + j, zero);
      if (whole + tid < V) Vec<T>::store1(dz + whole + tid, 0.f);
    }
    return;
  }
  const float k = p.inv_temp * kLog2e;
  Softmax s = {-__builtin_inff(), 0.f};
  for (int j = tid * N; j < whole; j += THREADS * N) {
    float x[N];
    Vec<T>::load(z + j, x);
    float m = s.max;
#pragma unroll
    for (int e = 0; e < N; ++e) m = __builtin_fmaxf(m, x[e]);
    s.sum *= rescale(s.max, m, k);
    s.max = m;
#pragma unroll
    for (int e = 0; e < N; ++e) s.sum += x[e] == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f((x[e] - m) * k);
  }
  if (whole + tid < V) {
    const float x = Vec<T>::load1(z + whole + tid);
    s = join(s, {x, x == -__builtin_inff() ? 0.f : (x - x) + 1.f}, k);   // (x - x: NaN where x is not finite)
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) s = join(s, {__shfl_xor(s.max, d), __shfl_xor(s.sum, d)}, k);
  if ((tid & 63) == 0) lds[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < WAVES; ++i) s = join(s, lds[i], k);
    out = row_terms(s, Vec<T>::load1(z + label), w, row, p);
  }
  __syncthreads();
  if constexpr (GRAD) {
    const RowOut o = out;
    const float f = -o.coef * o.inv_sum;
    const int y = (int)label;
    for (int j = tid * N; j < whole; j += THREADS * N) {
      float x[N];
      Vec<T>::load(z + j, x);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        x[e] = f * __builtin_amdgcn_exp2f((x[e] - o.max) * k);
        if (j + e == y) x[e] += o.coef;
      }
      Vec<T>::store(dz + j, x);
    }
    if (whole + tid < V) {
      const int j = whole + tid;
      float x = f * __builtin_amdgcn_exp2f((Vec<T>::load1(z + j) - o.max) * k);
      if (j == y) x += o.coef;
      Vec<T>::store1(dz + j, x);
    }
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

template <typename T>
hipError_t launch_policy_t(const himuon_policy &c, const PolicyParams &p, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  T *dz = reinterpret_cast<T *>(c.dlogits);
  // (a grid's x extent holds 2^31 - 1 blocks; rows beyond go into further launches)
  constexpr int64_t kRows = (int64_t)1 << 30;
  for (int64_t r = 0; r < c.rows; r += kRows) {
    const dim3 grid((unsigned)(c.rows - r < kRows ? c.rows - r : kRows));
    PolicyParams q = p;
    q.label += r;
    q.weight += r;
    q.advantage += r;
    if (q.old_logp) q.old_logp += r;
    if (q.ref_logp) q.ref_logp += r;
    q.logp += r;
    q.part += 3 * r;
    const T *zr = z + r * c.ld_logits;
    if (dz)
      hipLaunchKernelGGL((policy_row_kernel<T, true>), grid, dim3(THREADS), 0, stream, zr, dz + r * c.ld_dlogits, q);
    else
      hipLaunchKernelGGL((policy_row_kernel<T, false>), grid, dim3(THREADS), 0, stream, zr, nullptr, q);
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
  p.inv_temp = (float)(1.0 / c.temperature);
  p.low = (float)(1.0 - c.clip_low);
  p.high = (float)(1.0 + c.clip_high);
  p.kl_coef = (float)c.kl_coef;
  p.grad_scale = (float)c.grad_scale;
  return c.dtype == HIMUON_BF16 ? launch_policy_t<__bf16>(c, p, stream) : launch_policy_t<float>(c, p, stream);
}

}  // namespace himuon
