// Clipped policy loss with a KL term over sampled tokens, forward and gradient
// (himuon_policy_loss): a row softmax, a few scalars per row, and the gradient row.
//
// All sums, maxima and exponents are fp32 (the joined sums over rows fp64); the only
// rounding to fewer bits is that of the gradient to bf16 logits' own type.
#include "device_common.h"
#include "himuon_internal.h"
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

// Constants of a call in fp32.
struct PolicyParams {
  const int64_t *label;
  const float *weight, *advantage, *old_logp, *ref_logp;
  float *logp;
  f32x4 *part;        // workspace: per row, weight times (-min(u, c), kl, clipped, 0)
  f32x2 *spans;       // workspace, of rows that are cut into spans instead: per row and span, the span's
                      // largest logit and its sum; then the row's label's logit
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
template <class T, bool ZY = true>   // (ZY false: all but zy, and z is not used)
__device__ __forceinline__ RowIn row_in(const T *z, int64_t row, const PolicyParams &p) {
  RowIn r;
  r.w = gmem(p.weight)[row];
  const int64_t y = gmem(p.label)[row];
  r.label = r.w != 0.f && y >= 0 && y < p.vocab ? (int32_t)y : -1;
  if (r.label < 0) return r;
  r.adv = gmem(p.advantage)[row];
  r.old = p.old_logp ? gmem(p.old_logp)[row] : 0.f;
  r.ref_logp = p.ref_logp ? gmem(p.ref_logp)[row] : 0.f;
  if constexpr (ZY) r.zy = Vec<T>::load1(z + r.label);
  return r;
}

// A row's log probability, loss terms (weight times -min(u, c), kl and clipped), and its
// gradient's factor of (j == label) - p_j.
struct RowTerms {
  float lp, coef;
  f32x4 part;
};
__device__ __forceinline__ RowTerms row_terms(Softmax s, const RowIn &r, const PolicyParams &p) {
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
  const float kl_part = p.kl_coef != 0.f ? p.kl_coef * em1 : 0.f;   // (an infinite KL that does not count)
  return {lp, ((clipped ? 0.f : -u) - kl_part) * r.w * p.grad_scale * p.inv_temp,
          f32x4{r.w * -(clipped ? c : u), r.w * (em1 - d), clipped ? r.w : 0.f, 0.f}};
}
__device__ __forceinline__ void write_terms(float lp, f32x4 part, int64_t row, const PolicyParams &p) {
  gmem(p.logp)[row] = lp;
  gmem(p.part)[row] = part;
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
// A vector of the gradient: coef ((j == label) - p_j), f = -coef / sum.
template <class T, bool NT>
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
  Vec<T>::template store<NT>(p, x);
}

template <class T, int THR, bool NT>
__device__ __forceinline__ void zero_row(T *dz, int V) {
  constexpr int N = Vec<T>::N;
  const float zero[N] = {};
  const int whole = V / N * N;
  for (int j = threadIdx.x * N; j < whole; j += THR * N) Vec<T>::template store<NT>(dz + j, zero);
  if (whole + (int)threadIdx.x < V) Vec<T>::store1(dz + whole + threadIdx.x, 0.f);
}

// What a kernel writes besides a row's terms: nothing, the gradient, or the gradient past the
// caches.
enum { kForward = 0, kGradient = 1, kGradientNT = 2 };

// One block per row, the row in registers: K vectors of 16 bytes a thread, and one element
// of the row's last V % N on the first threads.  The row is read once and the gradient
// written once; -inf stands in for what lies beyond the row.
template <typename T, int THR, int K, int OUT>
__global__ __launch_bounds__(THR) void policy_row_kernel(const T *logits, T *dlogits, PolicyParams p) {
  constexpr int N = Vec<T>::N;
  constexpr bool GRAD = OUT != kForward, NT = OUT == kGradientNT;
  __shared__ Softmax lds[THR / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, V = p.vocab, vecs = V / N, rest = vecs * N + tid;
  const T *z = logits + row * p.ld_logits;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const RowIn r = row_in(z, row, p);
  if (r.label < 0) {
    if (tid == 0) write_terms(0.f, f32x4{0.f, 0.f, 0.f, 0.f}, row, p);
    if constexpr (GRAD) zero_row<T, THR, NT>(dz, V);
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
  const RowTerms t = row_terms(s, r, p);
  const float coef = t.coef;
  if (tid == 0) write_terms(t.lp, t.part, row, p);
  if constexpr (GRAD) {
    const float f = -coef / s.sum;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int j = (tid + i * THR) * N;
      if (tid + i * THR < vecs) gradient<T, NT>(dz + j, v[i], p.k, s.ref, f, coef, r.label - j);
    }
    if (rest < V) Vec<T>::store1(dz + rest, f * pow2(tail, p.k, s.ref) + (rest == r.label ? coef : 0.f));
  }
}

// Rows that do not fit in a block's registers: as many vectors as fit are held, the others
// are read again for the gradient, in the reverse order, mostly from the last-level cache
// (one block of 1024 threads a CU keeps the rows in flight below its 256 MB).  The forward
// pass alone holds nothing and runs two blocks a CU.  1000 fp32 rows of 128256, 1 in 5 left
// out: gradient 212 us held, 263 us with every vector read twice (193 us with the stores past
// the L2s, 4.8 TB/s of what has to move); forward 90 us held, 78 us streamed.
constexpr int kLongThreads = 1024, kHeldVecs = 1024 * 16;   // vectors that a block's registers hold
template <int OUT>
constexpr int kLongK = OUT != kForward ? 16 : 0;
template <typename T, int OUT>
__global__ __launch_bounds__(kLongThreads) void policy_long_kernel(const T *logits, T *dlogits, PolicyParams p) {
  constexpr int N = Vec<T>::N, THR = kLongThreads, K = kLongK<OUT>;
  constexpr bool GRAD = OUT != kForward, NT = OUT == kGradientNT;
  __shared__ Softmax lds[THR / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, V = p.vocab, vecs = V / N, rest = vecs * N + tid;
  const T *z = logits + row * p.ld_logits;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const RowIn r = row_in(z, row, p);
  if (r.label < 0) {
    if (tid == 0) write_terms(0.f, f32x4{0.f, 0.f, 0.f, 0.f}, row, p);
    if constexpr (GRAD) zero_row<T, THR, NT>(dz, V);
    return;
  }
  u32x4 v[K > 0 ? K : 1];
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = Vec<T>::load(z + (tid + i * THR) * N);   // the row is longer than these
  const float tail = rest < V ? Vec<T>::load1(z + rest) : -__builtin_inff();
  float m = tail;
#pragma unroll
  for (int i = 0; i < K; ++i) m = max_of<T>(v[i], m);
  float ref = ref_of(m), sum = pow2(tail, p.k, ref);
#pragma unroll
  for (int i = 0; i < K; ++i) {
    hold_packed(v[i]);
    sum += sum_of<T>(v[i], p.k, ref);
    hold_packed(v[i]);
  }
  int at = tid + K * THR;
  for (; at < vecs; at += THR) {
    const u32x4 x = Vec<T>::load(z + (int64_t)at * N);
    m = max_of<T>(x, m);
    const float to = ref_of(m);
    sum = (sum > 0.f ? sum * pow2(ref, p.k, to) : sum) + sum_of<T>(x, p.k, to);
    ref = to;
  }
  const Softmax s = block_softmax<THR / 64>(m, sum, p.k, lds);
  const RowTerms t = row_terms(s, r, p);
  const float coef = t.coef;
  if (tid == 0) write_terms(t.lp, t.part, row, p);
  if constexpr (GRAD) {
    const float f = -coef / s.sum;
    for (at -= THR; at >= K * THR; at -= THR)
      gradient<T, NT>(dz + (int64_t)at * N, Vec<T>::load(z + (int64_t)at * N), p.k, s.ref, f, coef, r.label - at * N);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int j = (tid + i * THR) * N;
      gradient<T, NT>(dz + j, v[i], p.k, s.ref, f, coef, r.label - j);
    }
    if (rest < V) Vec<T>::store1(dz + rest, f * pow2(tail, p.k, s.ref) + (rest == r.label ? coef : 0.f));
  }
}

// The block's sums of part over its threads, in fp64 and a fixed order, written as stats by
// thread 0.  W waves; every thread calls it.
template <int W>
__device__ __forceinline__ void write_stats(const double (&mine)[3], float kl_coef, float *stats) {
  __shared__ double lds[W][3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const double s = wave_sum(mine[k]);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6][k] = s;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  double t[3] = {0, 0, 0};
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int k = 0; k < 3; ++k) t[k] += lds[i][k];
  gmem(stats)[0] = (float)(kl_coef != 0.f ? t[0] + (double)kl_coef * t[1] : t[0]);
#pragma unroll
  for (int k = 0; k < 3; ++k) gmem(stats)[1 + k] = (float)t[k];
}

__global__ __launch_bounds__(1024) void policy_join_kernel(const f32x4 *part, int64_t rows, float kl_coef,
                                                           float *stats) {
  double s[3] = {0, 0, 0};
  constexpr int U = 8;   // rows a thread has in flight
  for (int64_t i = threadIdx.x; i < rows; i += 1024 * U) {
    f32x4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (i + u * 1024 < rows) x[u] = gmem(part)[i + u * 1024];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 3; ++k) s[k] += (double)x[u][k];
  }
  write_stats<16>(s, kl_coef, stats);
}

// Few long rows: a row's vectors are cut into spans of kSpanVecs, one block each, so that a
// handful of rows still occupies the whole chip.  The first kernel leaves each span's largest
// logit and sum, and the row's label's logit; in the second one every block joins its row's
// spans (one per lane and turn) and writes its span of the gradient, and one block more computes
// the rows' terms and stats.  The span of a row's last V % N elements is its last one.
// A gradient may be written over its logits, and the second kernel's blocks run in any order: no
// block of it reads a logit outside its own span, so the label's logit comes from the first.  It
// stands behind the spans, where a join's loads reach it in the same turn.
constexpr int kSpanThreads = 256, kSpanK = 4, kSpanVecs = kSpanThreads * kSpanK;
constexpr int64_t span_count(int64_t vecs) { return vecs < 1 ? 1 : (vecs + kSpanVecs - 1) / kSpanVecs; }

template <typename T>
__global__ __launch_bounds__(kSpanThreads) void policy_span_kernel(const T *logits, PolicyParams p) {
  constexpr int N = Vec<T>::N, THR = kSpanThreads;
  __shared__ Softmax lds[THR / 64];
  const int64_t row = blockIdx.y;
  const int tid = threadIdx.x, V = p.vocab, vecs = V / N, v0 = blockIdx.x * kSpanVecs, rest = vecs * N + tid;
  const T *z = logits + row * p.ld_logits;
  const float w = gmem(p.weight)[row];
  const int64_t y = gmem(p.label)[row];
  if (!(w != 0.f && y >= 0 && y < V)) return;
  const float zy = Vec<T>::load1(z + y);   // (by every block: a branch would wait for it before the vectors)
  u32x4 v[kSpanK];
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) {
    const int at = v0 + tid + i * THR;
    v[i] = u32x4{Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest};
    if (at < vecs) v[i] = Vec<T>::load(z + (int64_t)at * N);
  }
  const bool has_rest = blockIdx.x == gridDim.x - 1 && rest < V;
  const float tail = has_rest ? Vec<T>::load1(z + rest) : -__builtin_inff();
  float m = tail;
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) m = max_of<T>(v[i], m);
  const float ref = ref_of(m);
  float sum = pow2(tail, p.k, ref);
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) sum += sum_of<T>(v[i], p.k, ref);
  const Softmax s = block_softmax<THR / 64>(m, sum, p.k, lds);
  // (a span of nothing but -inf has ref 0 and sum 0: its largest logit is -inf)
  if (tid == 0) {
    f32x2 *out = p.spans + row * (gridDim.x + 1);
    gmem(out)[blockIdx.x] = f32x2{s.sum == 0.f ? -__builtin_inff() : s.ref, s.sum};
    if (blockIdx.x == 0) gmem(out)[gridDim.x] = f32x2{zy, 0.f};
  }
}

// A row's softmax from its n spans (1 at least), and its label's logit; every lane of a wave
// calls it.
__device__ __forceinline__ Softmax join_spans(const f32x2 *spans, int n, float k, float &label_logit) {
  const int lane = threadIdx.x & 63;
  Softmax s = {0.f, 0.f};
  float top = -__builtin_inff();
  int i = 0;
  do {   // (with a loop of no turn the compiler waits for the caller's vectors again between their stores: 0.5 us)
    f32x2 x = {-__builtin_inff(), 0.f};
    if (i + lane <= n) x = gmem(spans)[i + lane];
    if (n - i < 64) {
      label_logit = __shfl(x[0], n - i);
      if (i + lane == n) x = f32x2{-__builtin_inff(), 0.f};
    }
    const float m = __builtin_fmaxf(top, wave_max(x[0])), to = ref_of(m);
    const float part = wave_sum(x[1] * pow2(x[0], k, to));
    s.sum = (s.sum > 0.f ? s.sum * pow2(s.ref, k, to) : s.sum) + part;
    s.ref = to;
    top = m;
    i += 64;
  } while (i <= n);
  return s;
}

// The same for a row on four neighbouring lanes, so that one block takes 64 rows at a time:
// each lane joins every fourth span, eight loads in flight, and the four are joined.
constexpr int kRowLanes = 4;
__device__ __forceinline__ Softmax join_spans_quad(const f32x2 *spans, int n, float k, float &label_logit) {
  constexpr int U = 8;
  label_logit = gmem(spans)[n][0];
  float top = -__builtin_inff();
  Softmax s = {0.f, 0.f};
  for (int i = threadIdx.x % kRowLanes; i < n; i += kRowLanes * U) {
    f32x2 x[U];
    float m = top;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = f32x2{-__builtin_inff(), 0.f};
      if (i + u * kRowLanes < n) x[u] = gmem(spans)[i + u * kRowLanes];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) m = __builtin_fmaxf(m, x[u][0]);
    const float to = ref_of(m);
    s.sum = s.sum > 0.f ? s.sum * pow2(s.ref, k, to) : s.sum;
#pragma unroll
    for (int u = 0; u < U; ++u) s.sum += x[u][1] * pow2(x[u][0], k, to);
    s.ref = to;
    top = m;
  }
#pragma unroll
  for (int d = 1; d < kRowLanes; d *= 2) {
    const float m = __builtin_fmaxf(top, __shfl_xor(top, d)), to = ref_of(m);
    s.sum *= pow2(top, k, to);   // (a lane without spans has sum 0 and power 0)
    s.sum += __shfl_xor(s.sum, d);
    s.ref = to;
    top = m;
  }
  return s;
}

template <typename T>
__global__ __launch_bounds__(kSpanThreads) void policy_span_finish_kernel(const T *logits, T *dlogits, PolicyParams p,
                                                                          int32_t rows, int32_t spans, float *stats) {
  constexpr int N = Vec<T>::N, THR = kSpanThreads;
  const int tid = threadIdx.x, V = p.vocab, vecs = V / N;
  if (blockIdx.y == 0) {   // first in the grid, for it takes longest (without a gradient it is the grid)
    if (blockIdx.x != 0) return;
    double sum[3] = {0, 0, 0};
    for (int row = tid / kRowLanes; row < rows; row += THR / kRowLanes) {
      RowIn r = row_in<T, false>(nullptr, row, p);
      RowTerms t = {0.f, 0.f, f32x4{0.f, 0.f, 0.f, 0.f}};
      if (r.label >= 0) {
        const Softmax s = join_spans_quad(p.spans + (int64_t)row * (spans + 1), spans, p.k, r.zy);
        t = row_terms(s, r, p);
      }
      if (tid % kRowLanes == 0) {
        gmem(p.logp)[row] = t.lp;
#pragma unroll
        for (int k = 0; k < 3; ++k) sum[k] += (double)t.part[k];
      }
    }
    write_stats<THR / 64>(sum, p.kl_coef, stats);
    return;
  }
  const int64_t row = blockIdx.y - 1;
  const int v0 = blockIdx.x * kSpanVecs, rest = vecs * N + tid;
  const bool has_rest = (int)blockIdx.x == spans - 1 && rest < V;
  const T *z = logits + row * p.ld_logits;
  T *dz = dlogits + row * p.ld_dlogits;
  RowIn r = row_in<T, false>(nullptr, row, p);
  if (r.label < 0) {
    const float zero[N] = {};
#pragma unroll
    for (int i = 0; i < kSpanK; ++i) {
      const int at = v0 + tid + i * THR;
      if (at < vecs) Vec<T>::template store<false>(dz + (int64_t)at * N, zero);
    }
    if (has_rest) Vec<T>::store1(dz + rest, 0.f);
    return;
  }
  u32x4 v[kSpanK];
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) {
    const int at = v0 + tid + i * THR;
    v[i] = u32x4{0, 0, 0, 0};
    if (at < vecs) v[i] = Vec<T>::load(z + (int64_t)at * N);
  }
  const float tail = has_rest ? Vec<T>::load1(z + rest) : 0.f;
  const Softmax s = join_spans(p.spans + row * (spans + 1), spans, p.k, r.zy);
  const float coef = row_terms(s, r, p).coef, f = -coef / s.sum;
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) {
    const int at = v0 + tid + i * THR;
    if (at < vecs) gradient<T, false>(dz + (int64_t)at * N, v[i], p.k, s.ref, f, coef, r.label - at * N);
  }
  if (has_rest) Vec<T>::store1(dz + rest, f * pow2(tail, p.k, s.ref) + (rest == r.label ? coef : 0.f));
}

// Measured on graphs of 21 calls, split against one block a row, gradient included (us), rows x
// vocabulary.  bf16: 1 x 50257 5.6 / 10.6, 8 x 131072 6.2 / 17.9, 64 x 4096 5.7 / 5.8, 64 x 50257
// 9.5 / 12.6, 96 x 4096 6.9 / 5.9, 96 x 128256 15.0 / 21.2, 128 x 16384 7.5 / 7.4, 128 x 128256
// 18.0 / 20.1, 192 x 50257 15.4 / 15.5, 192 x 128256 26.4 / 23.1.  fp32: 1 x 50257 5.9 / 9.8, 8 x
// 131072 6.7 / 19.5, 64 x 4096 6.1 / 5.6, 64 x 16384 6.7 / 7.0, 64 x 131072 16.9 / 23.2, 65 x 128256
// 17.9 / 22.3, 80 x 128256 21.6 / 23.1, 96 x 16384 9.3 / 7.9, 96 x 128256 26.0 / 24.8, 128 x 16384
// 10.0 / 8.5, 128 x 128256 38.2 / 28.6.  One rule for both types, which suits bf16 throughout and
// fp32 up to 64 rows; of 65 to 128 fp32 rows it suits the forward pass (80 x 128256 13.2 / 18.2, 128
// x 60000 11.3 / 10.5) and the longest ones.
constexpr int kFewRows = 128;
bool few_rows(int64_t rows, int64_t vecs) {
  return rows > 0 && ((rows <= 64 && vecs >= 256) || (rows <= kFewRows && vecs >= 2048));
}

// A gradient that the L2s together (32 MB) cannot hold goes past them: 4096 x 128256 bf16 356 /
// 339 us, 256 x 128256 33 / 28 us, 1000 x 128256 fp32 213 / 195 us.  A smaller one stays for
// whoever reads it next.
constexpr double kL2Bytes = 32e6;

template <typename T, int THR, int K>
void launch_rows(const T *z, T *dz, unsigned rows, int out, const PolicyParams &p, hipStream_t stream) {
  const dim3 grid(rows), block(THR);
  if (out == kForward) hipLaunchKernelGGL((policy_row_kernel<T, THR, K, kForward>), grid, block, 0, stream, z, dz, p);
  else if (out == kGradient) hipLaunchKernelGGL((policy_row_kernel<T, THR, K, kGradient>), grid, block, 0, stream, z, dz, p);
  else hipLaunchKernelGGL((policy_row_kernel<T, THR, K, kGradientNT>), grid, block, 0, stream, z, dz, p);
}
template <typename T>
void launch_long_rows(const T *z, T *dz, unsigned rows, int out, const PolicyParams &p, hipStream_t stream) {
  const dim3 grid(rows), block(kLongThreads);
  // (fewer rows are cut into spans: the gradient is one that the L2s cannot hold)
  static_assert((kFewRows + 1.0) * kHeldVecs * 16 > kL2Bytes, "long rows past the L2s");
  if (out == kForward) hipLaunchKernelGGL((policy_long_kernel<T, kForward>), grid, block, 0, stream, z, dz, p);
  else hipLaunchKernelGGL((policy_long_kernel<T, kGradientNT>), grid, block, 0, stream, z, dz, p);
}

template <typename T>
hipError_t launch_policy_t(const himuon_policy &c, const PolicyParams &p, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  T *dz = reinterpret_cast<T *>(c.dlogits);
  const int64_t vecs = c.vocab / Vec<T>::N;
  if (few_rows(c.rows, vecs)) {
    const unsigned spans = (unsigned)span_count(vecs), rows = (unsigned)c.rows;
    hipLaunchKernelGGL((policy_span_kernel<T>), dim3(spans, rows), dim3(kSpanThreads), 0, stream, z, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // without a gradient: the block of the stats alone
    hipLaunchKernelGGL((policy_span_finish_kernel<T>), dz ? dim3(spans, rows + 1) : dim3(1, 1), dim3(kSpanThreads), 0,
                       stream, z, dz, p, (int32_t)rows, (int32_t)spans, c.stats);
    return hipGetLastError();
  }
  const int out = !dz ? kForward : (double)c.rows * c.vocab * sizeof(T) > kL2Bytes ? kGradientNT : kGradient;
  constexpr int64_t kRows = (int64_t)1 << 21;   // a launch: a grid holds fewer than 2^32 threads
  for (int64_t r = 0; r < c.rows; r += kRows) {
    const unsigned rows = (unsigned)(c.rows - r < kRows ? c.rows - r : kRows);
    PolicyParams q = p;
    q.label += r;
    q.weight += r;
    q.advantage += r;
    if (q.old_logp) q.old_logp += r;
    if (q.ref_logp) q.ref_logp += r;
    q.logp += r;
    q.part += r;
    const T *zr = z + r * c.ld_logits;
    T *dr = dz ? dz + r * c.ld_dlogits : nullptr;
    if (vecs <= 64 * 4) launch_rows<T, 64, 4>(zr, dr, rows, out, q, stream);
    else if (vecs <= 256 * 4) launch_rows<T, 256, 4>(zr, dr, rows, out, q, stream);
    else if (vecs <= 512 * 4) launch_rows<T, 512, 4>(zr, dr, rows, out, q, stream);
    else if (vecs <= 512 * 8) launch_rows<T, 512, 8>(zr, dr, rows, out, q, stream);
    else if (vecs <= 1024 * 8) launch_rows<T, 1024, 8>(zr, dr, rows, out, q, stream);
    else if (vecs <= kHeldVecs) launch_rows<T, 1024, 16>(zr, dr, rows, out, q, stream);
    else launch_long_rows<T>(zr, dr, rows, out, q, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(policy_join_kernel, dim3(1), dim3(1024), 0, stream, p.part, c.rows, p.kl_coef, c.stats);
  return hipGetLastError();
}

}  // namespace

// The spans of few long rows and their labels' logits, or the rows' terms.
size_t policy_workspace(const himuon_policy &p) {
  const int64_t vecs = p.vocab / (p.dtype == HIMUON_BF16 ? 8 : 4);
  return (size_t)p.rows * (few_rows(p.rows, vecs) ? (span_count(vecs) + 1) * sizeof(f32x2) : sizeof(f32x4));
}

hipError_t launch_policy(const himuon_policy &c, void *workspace, hipStream_t stream) {
  PolicyParams p{};
  p.label = c.label;
  p.weight = c.weight;
  p.advantage = c.advantage;
  p.old_logp = c.old_logp;
  p.ref_logp = c.ref_logp;
  p.logp = c.logp;
  p.part = reinterpret_cast<f32x4 *>(workspace);
  p.spans = reinterpret_cast<f32x2 *>(workspace);
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
