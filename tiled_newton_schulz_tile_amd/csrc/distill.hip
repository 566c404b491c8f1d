// Distillation from a teacher's top logits, forward and gradient (himuon_distill_loss): the
// Kullback-Leibler divergence from a teacher who names k tokens a row, and perhaps one class of
// all others, to the student's softmax.
//
// With named tokens (those of the teacher's entries) and the rest, a row is two softmaxes that
// share one pass over the logits.  The rest's largest logit and sum are kept apart from the
// named tokens' ones: the probability that the student gives to all of the rest is then as exact
// where it is 1e-30 as where it is one half, which 1 minus the named tokens' probabilities is not.
// A bitmap of the row in LDS says which logits are named; those are taken out of the row's
// vectors (-inf in their place) and come from the entries instead, a few a row.
//
// All sums, maxima and exponents are fp32 (the sum over rows fp64); the only rounding to fewer
// bits is that of the gradient to bf16 logits' own type.
#include "device_common.h"
#include "himuon_internal.h"
#include "row_softmax.h"

namespace himuon {
namespace {

// Constants of a call in fp32.
struct DistillParams {
  const void *value;
  const int64_t *index;
  const float *rest, *weight;
  float *kl;
  unsigned *ticket;   // workspace, of rows that are cut into spans: counts the rows that are done,
  f32x4 *spans;       // per row and span the rest's and the named tokens' largest logit and sum,
  float *entry_z;     // and the student's logit of every entry
  int64_t ld_logits, ld_dlogits, ld_top;
  int32_t vocab, entries, value_bf16;
  float k;            // log2(e) / temperature
  float inv_temp;     // 1 / temperature
  float coef;         // grad_scale / temperature
};

constexpr int kNone = -1;   // an entry that does not count

// A row's entries in LDS, and the bitmap of the tokens that they name.
struct EntryLds {
  int *token;        // kNone, or the token
  float *t, *z;      // the teacher's logit over the temperature, the student's logit
  unsigned *bits;
  int *twice;        // not 0: some token is named more than once
};
__device__ __forceinline__ EntryLds entry_lds(unsigned *lds, int entries) {
  return {reinterpret_cast<int *>(lds) + 1, reinterpret_cast<float *>(lds) + 1 + entries,
          reinterpret_cast<float *>(lds) + 1 + 2 * entries, lds + 1 + 3 * entries, reinterpret_cast<int *>(lds)};
}
size_t entry_lds_bytes(int64_t bits, int entries) { return (1 + 3 * (size_t)entries + (size_t)(bits + 31) / 32) * 4; }

__device__ __forceinline__ float entry_value(const DistillParams &p, int64_t at) {
  return p.value_bf16 ? bf16_bits_to_f32(gmem(reinterpret_cast<const unsigned short *>(p.value))[at])
                      : gmem(reinterpret_cast<const float *>(p.value))[at];
}

// Entry j as it counts: each sum over named tokens takes a token once, at its first entry.
__device__ __forceinline__ bool first_of_token(const EntryLds &e, int j, int token, bool twice) {
  if (token == kNone) return false;
  if (twice)
    for (int i = 0; i < j; ++i)
      if (e.token[i] == token) return false;
  return true;
}

// The bits of a vector's elements; -inf in the place of those that are set.
template <class T>
__device__ __forceinline__ unsigned vector_bits(const unsigned *bits, int vec) {
  const unsigned b = reinterpret_cast<const unsigned char *>(bits)[Vec<T>::N == 8 ? vec : vec >> 1];
  return Vec<T>::N == 8 ? b : b >> 4 * (vec & 1) & 15u;
}
template <class T>
__device__ __forceinline__ void hide(u32x4 &v, unsigned b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned x = v[i];
    if constexpr (Vec<T>::N == 8) {
      if (b >> 2 * i & 1) x = (x & 0xffff0000u) | 0xff80u;
      if (b >> (2 * i + 1) & 1) x = (x & 0xffffu) | 0xff800000u;
    } else {
      if (b >> i & 1) x = 0xff800000u;
    }
    v[i] = x;
  }
}

// A softmax in parts: the largest logit (-inf: none) and the sum of powers of the distances to it.
struct Part {
  float max, sum;
};
__device__ __forceinline__ void add(Part &s, float z, float k) {
  const float m = __builtin_fmaxf(s.max, z), to = ref_of(m);
  s.sum = s.sum * pow2(s.max, k, to) + pow2(z, k, to);
  s.max = m;
}
__device__ __forceinline__ Part join(Part a, Part b, float k) {
  const float m = __builtin_fmaxf(a.max, b.max), to = ref_of(m);
  return {m, a.sum * pow2(a.max, k, to) + b.sum * pow2(b.max, k, to)};
}
__device__ __forceinline__ Part wave_join(Part s, float k) {
  const float m = wave_max(s.max);
  return {m, wave_sum(s.sum * pow2(s.max, k, ref_of(m)))};
}
// M softmaxes over a block of W waves; lds holds W M entries.
template <int W, int M>
__device__ __forceinline__ void block_join(Part (&s)[M], const float (&k)[M], Part *lds) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    s[i] = wave_join(s[i], k[i]);
    if (W > 1 && lane == 0) lds[(threadIdx.x >> 6) * M + i] = s[i];
  }
  if constexpr (W == 1) return;
  lds_barrier();
#pragma unroll
  for (int i = 0; i < M; ++i) {
    s[i] = {-__builtin_inff(), 0.f};
    if (lane < W) s[i] = lds[lane * M + i];
    s[i] = wave_join(s[i], k[i]);
  }
}

// What a row's gradient and divergence need, the same in every thread.
struct RowCoefs {
  bool live;            // the teacher has some probability
  float ref, inv_sum, log_sum;     // the student's softmax over all tokens
  float teacher_ref, teacher_inv, teacher_log;
  float rest_ref, rest_f;          // a token u of the rest: gradient rest_f 2^((z_u - rest_ref) k)
  float coef;                      // of the row's gradient
  float rest_kl;                   // the rest's part of the divergence
};
__device__ __forceinline__ RowCoefs row_coefs(Part rest, Part named, Part teacher, float teacher_rest, float weight,
                                              const DistillParams &p) {
  RowCoefs r;
  r.live = !(teacher.max == -__builtin_inff() && teacher.sum == 0.f);
  const Part all = join(rest, named, p.k);
  r.ref = ref_of(all.max);
  r.inv_sum = 1.f / all.sum;
  r.log_sum = kLn2 * __builtin_amdgcn_logf(all.sum);
  r.teacher_ref = ref_of(teacher.max);
  r.teacher_inv = 1.f / teacher.sum;
  r.teacher_log = kLn2 * __builtin_amdgcn_logf(teacher.sum);
  const float q = pow2(teacher_rest, (float)kLog2e, r.teacher_ref) * r.teacher_inv;
  r.rest_ref = ref_of(rest.max);
  r.coef = weight * p.coef * (teacher.sum == teacher.sum ? 1.f : teacher.sum);
  float f = pow2(rest.max, p.k, r.ref) * r.inv_sum;
  r.rest_kl = 0.f;
  if (!(q <= 0.f)) {
    f -= rest.sum > 0.f ? q / rest.sum : 0.f;   // (a rest of probability 0 has a gradient of 0 and an infinite divergence)
    const float lp = rest.sum > 0.f ? (rest.max - r.ref) * p.inv_temp + kLn2 * __builtin_amdgcn_logf(rest.sum) - r.log_sum
                                    : rest.sum - __builtin_inff();
    r.rest_kl = q * ((teacher_rest - r.teacher_ref) - r.teacher_log - lp);
  }
  r.rest_f = r.coef * f;
  return r;
}
__device__ __forceinline__ float entry_q(float t, const RowCoefs &r) {
  return pow2(t, (float)kLog2e, r.teacher_ref) * r.teacher_inv;
}
// One wave: the row's divergence (every lane has it).
__device__ __forceinline__ float row_kl(const EntryLds &e, const RowCoefs &r, const DistillParams &p) {
  float kl = 0.f;
  for (int j = threadIdx.x & 63; j < p.entries; j += 64) {
    if (e.token[j] == kNone) continue;
    const float t = e.t[j], q = entry_q(t, r);
    if (q != 0.f) kl += q * ((t - r.teacher_ref) - r.teacher_log - ((e.z[j] - r.ref) * p.inv_temp - r.log_sum));
  }
  return wave_sum(kl) + r.rest_kl;
}
// The gradient of entry j's token: the entries of one token write the same value.
__device__ __forceinline__ float entry_gradient(const EntryLds &e, int j, bool twice, const RowCoefs &r,
                                                const DistillParams &p) {
  const int token = e.token[j];
  float q = 0.f;
  if (twice) {
    for (int i = 0; i < p.entries; ++i)
      if (e.token[i] == token) q += entry_q(e.t[i], r);
  } else {
    q = entry_q(e.t[j], r);
  }
  return r.coef * (pow2(e.z[j], p.k, r.ref) * r.inv_sum - q);
}
// A vector of the rest's gradient, but for the elements that are named.
template <class T, bool NT>
__device__ __forceinline__ void rest_gradient(T *dz, u32x4 v, unsigned b, const RowCoefs &r, float k) {
  constexpr int N = Vec<T>::N;
  float x[N];
  Vec<T>::unpack(v, x);
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = r.rest_f * pow2(x[e], k, r.rest_ref);
  if (b == 0) {
    Vec<T>::template store<NT>(dz, x);
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (!(b >> e & 1)) Vec<T>::store1(dz + e, x[e]);
}

enum { kForward = 0, kGradient = 1, kGradientNT = 2 };

// One block per row: K vectors of 16 bytes a thread are held in registers between the softmax and
// the gradient, and where the row is LONG the vectors behind them are read again for the gradient.
template <typename T, int THR, int K, bool LONG, int OUT>
__global__ __launch_bounds__(THR) void distill_row_kernel(const T *logits, T *dlogits, DistillParams p) {
  constexpr int N = Vec<T>::N;
  constexpr bool GRAD = OUT != kForward, NT = OUT == kGradientNT;
  extern __shared__ unsigned lds[];
  __shared__ Part parts[THR / 64 * 3];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, V = p.vocab, vecs = V / N, tail_at = vecs * N + tid;
  const T *z = logits + row * p.ld_logits;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const EntryLds e = entry_lds(lds, p.entries);
  const float w = gmem(p.weight)[row];
  if (w == 0.f) {
    if (tid == 0) gmem(p.kl)[row] = 0.f;
    if constexpr (GRAD) zero_row<T, THR, NT>(dz, V);
    return;
  }
  const float teacher_rest = p.rest ? gmem(p.rest)[row] : -__builtin_inff();
  int64_t token = kNone;   // of the thread's first entry
  float value = 0.f;
  if (tid < p.entries) {
    token = gmem(p.index)[row * p.ld_top + tid];
    value = entry_value(p, row * p.ld_top + tid);
  }
  u32x4 v[K > 0 ? K : 1];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    v[i] = u32x4{Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest};
    if (LONG || tid + i * THR < vecs) v[i] = Vec<T>::load(z + (tid + i * THR) * N);
  }
  float tail = tail_at < V ? Vec<T>::load1(z + tail_at) : -__builtin_inff();

  for (int i = tid; i < (V + 31) / 32; i += THR) e.bits[i] = 0;
  if (tid == 0) *e.twice = 0;
  lds_barrier();
  Part sums[3] = {{-__builtin_inff(), 0.f}, {-__builtin_inff(), 0.f}, {-__builtin_inff(), 0.f}};   // rest, named, teacher
  for (int j = tid; j < p.entries; j += THR) {
    if (j != tid) {
      token = gmem(p.index)[row * p.ld_top + j];
      value = entry_value(p, row * p.ld_top + j);
    }
    const bool counts = token >= 0 && token < V;
    e.token[j] = counts ? (int)token : kNone;
    if (!counts) continue;
    const float t = value * p.inv_temp;
    e.t[j] = t;
    e.z[j] = Vec<T>::load1(z + token);
    add(sums[2], t, (float)kLog2e);
    const unsigned bit = 1u << (token & 31);
    if (atomicOr(&e.bits[token >> 5], bit) & bit) *e.twice = 1;
  }
  lds_barrier();
  const bool twice = *e.twice != 0;
  if (tid == 0 && teacher_rest != -__builtin_inff()) add(sums[2], teacher_rest, (float)kLog2e);
  for (int j = tid; j < p.entries; j += THR)
    if (first_of_token(e, j, e.token[j], twice)) add(sums[1], e.z[j], p.k);
#pragma unroll
  for (int i = 0; i < K; ++i) {
    if (!LONG && tid + i * THR >= vecs) continue;
    const unsigned b = vector_bits<T>(e.bits, tid + i * THR);
    if (b) hide<T>(v[i], b);
  }
  const bool tail_named = tail_at < V && (e.bits[tail_at >> 5] >> (tail_at & 31) & 1);
  if (tail_named) tail = -__builtin_inff();

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
  if constexpr (LONG) {
    for (; at < vecs; at += THR) {
      u32x4 x = Vec<T>::load(z + (int64_t)at * N);
      const unsigned b = vector_bits<T>(e.bits, at);
      if (b) hide<T>(x, b);
      m = max_of<T>(x, m);
      const float to = ref_of(m);
      sum = (sum > 0.f ? sum * pow2(ref, p.k, to) : sum) + sum_of<T>(x, p.k, to);
      ref = to;
    }
  }
  sums[0] = {m, sum};
  const float ks[3] = {p.k, p.k, (float)kLog2e};
  block_join<THR / 64, 3>(sums, ks, parts);
  const RowCoefs r = row_coefs(sums[0], sums[1], sums[2], teacher_rest, w, p);
  if (!r.live) {
    if (tid == 0) gmem(p.kl)[row] = 0.f;
    if constexpr (GRAD) zero_row<T, THR, NT>(dz, V);
    return;
  }
  if (tid < 64) {
    const float kl = row_kl(e, r, p);
    if (tid == 0) gmem(p.kl)[row] = kl;
  }
  if constexpr (GRAD) {
    if constexpr (LONG) {
      for (at -= THR; at >= K * THR; at -= THR) {
        u32x4 x = Vec<T>::load(z + (int64_t)at * N);
        const unsigned b = vector_bits<T>(e.bits, at);
        if (b) hide<T>(x, b);
        rest_gradient<T, NT>(dz + (int64_t)at * N, x, b, r, p.k);
      }
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int vec = tid + i * THR;
      if (LONG || vec < vecs) rest_gradient<T, NT>(dz + vec * N, v[i], vector_bits<T>(e.bits, vec), r, p.k);
    }
    if (tail_at < V && !tail_named) Vec<T>::store1(dz + tail_at, r.rest_f * pow2(tail, p.k, r.rest_ref));
    for (int j = tid; j < p.entries; j += THR)
      if (e.token[j] != kNone) Vec<T>::store1(dz + e.token[j], entry_gradient(e, j, twice, r, p));
  }
}

// The sum over rows of weight times divergence, in fp64 and a fixed order; every thread of W waves
// calls it.  AGENT: other blocks of the launch wrote the divergences.
template <int W, bool AGENT>
__device__ __forceinline__ void write_loss(const float *weight, const float *kl, int64_t rows, float *loss) {
  __shared__ double lds[W];
  double s = 0;
  for (int64_t i = threadIdx.x; i < rows; i += W * 64) {
    float d;
    if constexpr (AGENT) d = __hip_atomic_load(&kl[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else d = gmem(kl)[i];
    if (d != 0.f) s += (double)gmem(weight)[i] * (double)d;
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = 0;
  for (int i = 0; i < W; ++i) s += lds[i];
  gmem(loss)[0] = (float)s;
}
__global__ __launch_bounds__(1024) void distill_join_kernel(const float *weight, const float *kl, int64_t rows, float *loss) {
  write_loss<16, false>(weight, kl, rows, loss);
}

// Few long rows: a row's vectors are cut into spans of kSpanVecs, one block each, so that a handful
// of rows still occupies the whole chip.  The first kernel leaves each span's two softmaxes and the
// logits of the entries that lie in it; in the second one every block joins its row's spans and
// writes its span of the gradient, and a row's first block its divergence.  The gradient may stand
// in the place of the logits: no block of the second kernel reads a logit outside its own span.
constexpr int kSpanThreads = 256, kSpanK = 4, kSpanVecs = kSpanThreads * kSpanK;
constexpr int64_t span_count(int64_t vecs) { return vecs < 1 ? 1 : (vecs + kSpanVecs - 1) / kSpanVecs; }

// A span's vectors and the row's last V % N elements, without the named ones, which are marked in
// the bitmap by their place in the span.
template <typename T>
struct Span {
  static constexpr int N = Vec<T>::N, THR = kSpanThreads, kBits = (kSpanVecs + 1) * N;
  int v0, vecs, first, end, tail_at;   // of the row's vectors and elements
  bool has_tail;
  u32x4 v[kSpanK];
  float tail;

  __device__ __forceinline__ Span(const T *z, int V, int spans) {
    const int tid = threadIdx.x;
    v0 = blockIdx.x * kSpanVecs;
    vecs = V / N;
    first = v0 * N;
    end = (int)blockIdx.x == spans - 1 ? V : first + kSpanVecs * N;
    tail_at = vecs * N + tid;
    has_tail = (int)blockIdx.x == spans - 1 && tail_at < V;
#pragma unroll
    for (int i = 0; i < kSpanK; ++i) {
      const int at = v0 + tid + i * THR;
      v[i] = u32x4{Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest};
      if (at < vecs) v[i] = Vec<T>::load(z + (int64_t)at * N);
    }
    tail = has_tail ? Vec<T>::load1(z + tail_at) : -__builtin_inff();
  }
  __device__ __forceinline__ void clear(const EntryLds &e) const {
    for (int i = threadIdx.x; i < (kBits + 31) / 32; i += THR) e.bits[i] = 0;
    if (threadIdx.x == 0) *e.twice = 0;
  }
  __device__ __forceinline__ bool holds(int64_t token) const { return token >= first && token < end; }
  // Marks token; a token that was marked already is named twice.
  __device__ __forceinline__ void mark(const EntryLds &e, int token) const {
    const unsigned bit = 1u << ((token - first) & 31);
    if (atomicOr(&e.bits[(token - first) >> 5], bit) & bit) *e.twice = 1;
  }
  __device__ __forceinline__ unsigned bits_of(const EntryLds &e, int i) const {
    return vector_bits<T>(e.bits, threadIdx.x + i * THR);
  }
  __device__ __forceinline__ bool tail_named(const EntryLds &e) const {
    return has_tail && (e.bits[(tail_at - first) >> 5] >> ((tail_at - first) & 31) & 1);
  }
  __device__ __forceinline__ void hide_named(const EntryLds &e) {
#pragma unroll
    for (int i = 0; i < kSpanK; ++i) {
      const unsigned b = bits_of(e, i);
      if (b) hide<T>(v[i], b);
    }
    if (tail_named(e)) tail = -__builtin_inff();
  }
};

template <typename T>
__global__ __launch_bounds__(kSpanThreads) void distill_span_kernel(const T *logits, DistillParams p) {
  constexpr int THR = kSpanThreads;
  extern __shared__ unsigned lds[];
  __shared__ Part parts[THR / 64 * 2];
  const int64_t row = blockIdx.y;
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && row == 0 && tid == 0) *p.ticket = 0;
  if (gmem(p.weight)[row] == 0.f) return;
  const T *z = logits + row * p.ld_logits;
  const EntryLds e = entry_lds(lds, p.entries);
  Span<T> s(z, p.vocab, gridDim.x);
  s.clear(e);
  lds_barrier();
  for (int j = tid; j < p.entries; j += THR) {
    const int64_t token = gmem(p.index)[row * p.ld_top + j];
    e.token[j] = s.holds(token) ? (int)token : kNone;
    if (!s.holds(token)) continue;
    s.mark(e, (int)token);
    e.z[j] = Vec<T>::load1(z + token);
    gmem(p.entry_z)[row * p.entries + j] = e.z[j];
  }
  lds_barrier();
  Part sums[2] = {{-__builtin_inff(), 0.f}, {-__builtin_inff(), 0.f}};
  const bool twice = *e.twice != 0;
  for (int j = tid; j < p.entries; j += THR)
    if (first_of_token(e, j, e.token[j], twice)) add(sums[1], e.z[j], p.k);
  s.hide_named(e);
  float m = s.tail;
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) m = max_of<T>(s.v[i], m);
  const float ref = ref_of(m);
  float sum = pow2(s.tail, p.k, ref);
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) sum += sum_of<T>(s.v[i], p.k, ref);
  sums[0] = {m, sum};
  const float ks[2] = {p.k, p.k};
  block_join<THR / 64, 2>(sums, ks, parts);
  if (tid == 0) gmem(p.spans)[row * gridDim.x + blockIdx.x] = f32x4{sums[0].max, sums[0].sum, sums[1].max, sums[1].sum};
}

// (without a gradient the grid has a row's first block alone)
template <typename T, bool GRAD>
__global__ __launch_bounds__(kSpanThreads) void distill_span_finish_kernel(const T *logits, T *dlogits, DistillParams p,
                                                                           int32_t spans, float *loss) {
  constexpr int THR = kSpanThreads, N = Vec<T>::N;
  extern __shared__ unsigned lds[];
  __shared__ Part parts[THR / 64];
  __shared__ bool joins;
  const int64_t row = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const EntryLds e = entry_lds(lds, p.entries);
  const float w = gmem(p.weight)[row];
  float kl = 0.f;
  if (w != 0.f || GRAD) {
    Span<T> s(logits + row * p.ld_logits, GRAD && w != 0.f ? p.vocab : 0, GRAD ? spans : 0);
    RowCoefs r;
    r.live = false;
    if (w != 0.f) {
      const float teacher_rest = p.rest ? gmem(p.rest)[row] : -__builtin_inff();
      s.clear(e);
      lds_barrier();
      Part teacher[1] = {{-__builtin_inff(), 0.f}};
      for (int j = tid; j < p.entries; j += THR) {
        const int64_t token = gmem(p.index)[row * p.ld_top + j];
        const bool counts = token >= 0 && token < p.vocab;
        e.token[j] = counts ? (int)token : kNone;
        if (!counts) continue;
        e.t[j] = entry_value(p, row * p.ld_top + j) * p.inv_temp;
        e.z[j] = gmem(p.entry_z)[row * p.entries + j];
        add(teacher[0], e.t[j], (float)kLog2e);
        if (GRAD && s.holds(token)) s.mark(e, (int)token);
      }
      if (tid == 0 && teacher_rest != -__builtin_inff()) add(teacher[0], teacher_rest, (float)kLog2e);
      Part rest = {-__builtin_inff(), 0.f}, named = rest;
      for (int i = lane; i < spans; i += 64) {
        const f32x4 x = gmem(p.spans)[row * spans + i];
        rest = join(rest, {x[0], x[1]}, p.k);
        named = join(named, {x[2], x[3]}, p.k);
      }
      rest = wave_join(rest, p.k);
      named = wave_join(named, p.k);
      const float ks[1] = {(float)kLog2e};
      block_join<THR / 64, 1>(teacher, ks, parts);
      r = row_coefs(rest, named, teacher[0], teacher_rest, w, p);
      if (r.live && blockIdx.x == 0 && tid < 64) kl = row_kl(e, r, p);
    }
    if constexpr (GRAD) {
      // (the span's own vectors were not read where the row is left out: its bounds are those of the call)
      const int v0 = blockIdx.x * kSpanVecs, vecs = p.vocab / N, tail_at = vecs * N + tid;
      const bool has_tail = (int)blockIdx.x == spans - 1 && tail_at < p.vocab;
      if (!r.live) {
        const float zero[N] = {};
#pragma unroll
        for (int i = 0; i < kSpanK; ++i) {
          const int at = v0 + tid + i * THR;
          if (at < vecs) Vec<T>::template store<false>(dz + (int64_t)at * N, zero);
        }
        if (has_tail) Vec<T>::store1(dz + tail_at, 0.f);
      } else {
        s.hide_named(e);
        const bool twice = *e.twice != 0;
#pragma unroll
        for (int i = 0; i < kSpanK; ++i) {
          const int at = v0 + tid + i * THR;
          if (at < vecs) rest_gradient<T, false>(dz + (int64_t)at * N, s.v[i], s.bits_of(e, i), r, p.k);
        }
        if (has_tail && !s.tail_named(e)) Vec<T>::store1(dz + tail_at, r.rest_f * pow2(s.tail, p.k, r.rest_ref));
        for (int j = tid; j < p.entries; j += THR)
          if (e.token[j] != kNone && s.holds(e.token[j])) Vec<T>::store1(dz + e.token[j], entry_gradient(e, j, twice, r, p));
      }
    }
  }
  if (blockIdx.x != 0) return;
  // the last row to finish (the ticket says which) joins all of them
  if (tid == 0) {
    __hip_atomic_store(&p.kl[row], kl, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    joins = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.y - 1;
  }
  __syncthreads();
  if (!joins) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  write_loss<THR / 64, true>(p.weight, p.kl, gridDim.y, loss);
}

constexpr int kFewRows = 128;
bool few_rows(int64_t rows, int64_t vecs) {
  return rows > 0 && ((rows <= 64 && vecs >= 256) || (rows <= kFewRows && vecs >= 2048));
}

// A gradient that the L2s together (32 MB) cannot hold goes past them.
constexpr double kL2Bytes = 32e6;

template <typename T, int THR, int K, bool LONG = false>
void launch_rows(const T *z, T *dz, unsigned rows, int out, const DistillParams &p, hipStream_t stream) {
  const dim3 grid(rows), block(THR);
  const size_t lds = entry_lds_bytes(p.vocab, p.entries);
  if (out == kForward) hipLaunchKernelGGL((distill_row_kernel<T, THR, LONG ? 0 : K, LONG, kForward>), grid, block, lds, stream, z, dz, p);
  else if (out == kGradient) hipLaunchKernelGGL((distill_row_kernel<T, THR, K, LONG, kGradient>), grid, block, lds, stream, z, dz, p);
  else hipLaunchKernelGGL((distill_row_kernel<T, THR, K, LONG, kGradientNT>), grid, block, lds, stream, z, dz, p);
}

template <typename T>
hipError_t launch_distill_t(const himuon_distill &c, const DistillParams &p, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  T *dz = reinterpret_cast<T *>(c.dlogits);
  const int64_t vecs = c.vocab / Vec<T>::N;
  if (few_rows(c.rows, vecs)) {
    const unsigned spans = (unsigned)span_count(vecs), rows = (unsigned)c.rows;
    const size_t lds = entry_lds_bytes(Span<T>::kBits, c.k);
    hipLaunchKernelGGL((distill_span_kernel<T>), dim3(spans, rows), dim3(kSpanThreads), lds, stream, z, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (dz)
      hipLaunchKernelGGL((distill_span_finish_kernel<T, true>), dim3(spans, rows), dim3(kSpanThreads), lds, stream, z, dz, p,
                         (int32_t)spans, c.loss);
    else
      hipLaunchKernelGGL((distill_span_finish_kernel<T, false>), dim3(1, rows), dim3(kSpanThreads), lds, stream, z, dz, p,
                         (int32_t)spans, c.loss);
    return hipGetLastError();
  }
  const int out = !dz ? kForward : (double)c.rows * c.vocab * sizeof(T) > kL2Bytes ? kGradientNT : kGradient;
  constexpr int64_t kRows = (int64_t)1 << 21;   // a launch: a grid holds fewer than 2^32 threads
  for (int64_t r = 0; r < c.rows; r += kRows) {
    const unsigned rows = (unsigned)(c.rows - r < kRows ? c.rows - r : kRows);
    DistillParams q = p;
    q.value = reinterpret_cast<const char *>(p.value) + r * p.ld_top * (p.value_bf16 ? 2 : 4);
    q.index += r * p.ld_top;
    q.weight += r;
    if (q.rest) q.rest += r;
    q.kl += r;
    const T *zr = z + r * c.ld_logits;
    T *dr = dz ? dz + r * c.ld_dlogits : nullptr;
    if (vecs <= 64 * 4) launch_rows<T, 64, 4>(zr, dr, rows, out, q, stream);
    else if (vecs <= 256 * 4) launch_rows<T, 256, 4>(zr, dr, rows, out, q, stream);
    else if (vecs <= 512 * 4) launch_rows<T, 512, 4>(zr, dr, rows, out, q, stream);
    else if (vecs <= 512 * 8) launch_rows<T, 512, 8>(zr, dr, rows, out, q, stream);
    else if (vecs <= 1024 * 8) launch_rows<T, 1024, 8>(zr, dr, rows, out, q, stream);
    else if (vecs <= 1024 * 16) launch_rows<T, 1024, 16>(zr, dr, rows, out, q, stream);
    else launch_rows<T, 1024, 16, true>(zr, dr, rows, out, q, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(distill_join_kernel, dim3(1), dim3(1024), 0, stream, p.weight, p.kl, c.rows, c.loss);
  return hipGetLastError();
}

}  // namespace

// The ticket, the spans of few long rows and their entries' logits; other rows need nothing.
size_t distill_workspace(const himuon_distill &p) {
  const int64_t vecs = p.vocab / (p.dtype == HIMUON_BF16 ? 8 : 4);
  return few_rows(p.rows, vecs) ? 16 + (size_t)p.rows * (span_count(vecs) * sizeof(f32x4) + p.k * sizeof(float)) : 0;
}

hipError_t launch_distill(const himuon_distill &c, void *workspace, hipStream_t stream) {
  DistillParams p{};
  p.value = c.value;
  p.index = c.index;
  p.rest = c.rest;
  p.weight = c.weight;
  p.kl = c.kl;
  const int64_t vecs = c.vocab / (c.dtype == HIMUON_BF16 ? 8 : 4);
  p.ticket = reinterpret_cast<unsigned *>(workspace);
  p.spans = reinterpret_cast<f32x4 *>(workspace) + 1;
  p.entry_z = reinterpret_cast<float *>(p.spans + c.rows * span_count(vecs));
  p.ld_logits = c.ld_logits;
  p.ld_dlogits = c.ld_dlogits;
  p.ld_top = c.ld_top;
  p.vocab = (int32_t)c.vocab;
  p.entries = c.k;
  p.value_bf16 = c.value_dtype == HIMUON_BF16;
  p.k = (float)(kLog2e / c.temperature);
  p.inv_temp = (float)(1.0 / c.temperature);
  p.coef = (float)(c.grad_scale / c.temperature);
  return c.dtype == HIMUON_BF16 ? launch_distill_t<__bf16>(c, p, stream) : launch_distill_t<float>(c, p, stream);
}

}  // namespace himuon
