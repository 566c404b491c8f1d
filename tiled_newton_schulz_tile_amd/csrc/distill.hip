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
// The rest's sums, maxima and exponents are fp32.  The gradient of a named token is a difference of
// two probabilities that may both be near 1: the few powers and sums that it takes are fp64, as is
// the sum over rows.  The only rounding to fewer bits is that of the gradient to bf16 logits' own
// type.
#include "device_common.h"
#include "himuon_internal.h"
#include "row_softmax.h"

namespace himuon {
namespace {

struct DistillParams {
  const void *value;
  const int64_t *index;
  const float *rest, *weight;
  float *kl;
  unsigned *ticket;   // workspace, of rows that are cut into spans: counts the rows that are done,
  f32x2 *spans;       // per row and span the rest's largest logit and sum,
  f32x2 *entry;       // and of every entry the student's logit, and 1 if it is the first of its token
  int64_t ld_logits, ld_dlogits, ld_top;
  int32_t vocab, entries, value_bf16;
  float k;                        // log2(e) / temperature
  float coef;                     // grad_scale / temperature
  double fine_k, temp, inv_temp;  // log2(e) / temperature, temperature, 1 / temperature
};

constexpr int kNone = -1;   // an entry that does not count

// A row's entries in LDS, what they sum to, and the bitmap of the tokens that they name: a byte for
// each vector of the row, at the place that marks() gives it.
struct EntrySums {
  unsigned named_max, teacher_max;   // ordered bits of the entries' largest logits; 0: none
  int twice;                         // not 0: some token is named more than once
  double named[16], teacher[16];     // sums of powers, by wave
};
struct EntryLds {
  int *token;        // kNone, or the token
  float *t, *z, *g;  // the teacher's logit, the student's logit, the gradient
  unsigned char *marks;
};
__device__ __forceinline__ EntryLds entry_lds(u32x4 *lds, size_t mark_bytes, int entries) {
  float *f = reinterpret_cast<float *>(reinterpret_cast<char *>(lds) + mark_bytes);
  return {reinterpret_cast<int *>(f), f + entries, f + 2 * entries, f + 3 * entries, reinterpret_cast<unsigned char *>(lds)};
}
constexpr size_t entry_lds_bytes(size_t mark_bytes, int entries) { return mark_bytes + 16 * (size_t)entries; }

__device__ __forceinline__ float entry_value(const DistillParams &p, int64_t at) {
  return p.value_bf16 ? bf16_bits_to_f32(gmem(reinterpret_cast<const unsigned short *>(p.value))[at])
                      : gmem(reinterpret_cast<const float *>(p.value))[at];
}
__device__ __forceinline__ unsigned ordered(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_ordered(unsigned o) {
  return __builtin_bit_cast(float, o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}
// The reference of a softmax from its largest logit's ordered bits (0 where there is none or it is
// -inf, whose powers are 0 then).
__device__ __forceinline__ float ordered_ref(unsigned o) { return o == 0 ? 0.f : ref_of(of_ordered(o)); }
// The teacher's, from its entries and its rest times the temperature.  That is fp64: its fp32 value may be thousands
// of octaves away, and beyond fp32's range.  (A NaN is in the sums.)
__device__ __forceinline__ double teacher_ref_of(unsigned o, double teacher_rest) {
  const double m = __builtin_fmax(o == 0 ? -__builtin_inf() : (double)of_ordered(o), teacher_rest);
  return m == -__builtin_inf() ? 0. : m;
}

// Marks element e of the vector whose byte is at `at`; one that is marked already is named twice.
__device__ __forceinline__ void mark(unsigned char *marks, int at, int e, EntrySums &sums) {
  const unsigned bit = 1u << (8 * (at & 3) + e);
  if (atomicOr(reinterpret_cast<unsigned *>(marks) + (at >> 2), bit) & bit) sums.twice = 1;
}
// Whether entry j stands for its token in sums over named tokens: the token's first entry does.
__device__ __forceinline__ bool first_of_token(const EntryLds &e, int j, bool twice) {
  if (twice)
    for (int i = 0; i < j; ++i)
      if (e.token[i] == e.token[j]) return false;
  return true;
}
// -inf in the place of the marked elements of a vector.
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

// The rest's softmax of a block of W waves from its threads' largest logits and sums.
template <int W>
__device__ __forceinline__ Softmax rest_join(float max, float sum, float k, Softmax *lds) {
  const int lane = threadIdx.x & 63;
  float m = wave_max(max);
  sum = wave_sum(sum * pow2(max, k, ref_of(m)));
  if (lane == 0) lds[threadIdx.x >> 6] = {m, sum};
  lds_barrier();
  const Softmax s = lds[lane % W];
  m = wave_max(s.ref);
  return {m, wave_sum(lane < W ? s.sum * pow2(s.ref, k, ref_of(m)) : 0.f)};
}

// A number that is the same in all lanes, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}

// What a row's gradient and divergence need, the same in every thread.
struct RowCoefs {
  bool live;                         // the teacher has some probability
  float named_ref;                   // of the entries' powers,
  double teacher_ref;                //   of the teacher's, and what these are multiplied with to be
  double named_f, teacher_f;         //   probabilities
  float ref;                         // the student's softmax over all tokens: the largest logit
  double sum, teacher_sum;           //   and the sum; the teacher's sum
  float rest_ref, rest_f;            // a token u of the rest: gradient rest_f 2^((z_u - rest_ref) k)
  float coef;                        // of the row's gradient
  bool rest_counts;                  // the teacher's rest has some probability
};
__device__ __forceinline__ double power(double z, double ref, const DistillParams &p) {
  return pow2_exact((z - ref) * p.fine_k);
}

// rest: the rest's largest logit (-inf: none) and sum; waves: those that left sums of entries;
// teacher_rest: times the temperature, as the teacher's logits are.
__device__ __forceinline__ RowCoefs row_coefs(Softmax rest, const EntrySums &sums, int waves, double teacher_rest,
                                              float weight, const DistillParams &p) {
  RowCoefs r;
  double named = 0, teacher = 0;
  for (int i = 0; i < waves; ++i) {
    named += sums.named[i];
    teacher += sums.teacher[i];
  }
  r.live = !(teacher == 0);
  r.named_ref = ordered_ref(sums.named_max);
  r.teacher_ref = teacher_ref_of(sums.teacher_max, teacher_rest);
  r.rest_ref = ref_of(rest.ref);
  const float named_max = named == 0 ? -__builtin_inff() : r.named_ref;
  r.ref = ref_of(__builtin_fmaxf(rest.ref, named_max));
  const double named_scale = power(named_max, r.ref, p), rest_scale = power(rest.ref, r.ref, p);
  r.sum = named * named_scale + (double)rest.sum * rest_scale;
  const double inv = 1. / r.sum;
  r.named_f = named_scale * inv;
  r.teacher_sum = teacher;
  r.teacher_f = 1. / teacher;
  const double q_rest = power(teacher_rest, r.teacher_ref, p) * r.teacher_f;
  r.rest_counts = !(q_rest <= 0);   // (NaN does)
  r.coef = weight * p.coef * (teacher == teacher ? 1.f : (float)teacher);
  float f = (float)(rest_scale * inv);
  // (a rest of probability 0 has a gradient of 0 and an infinite divergence)
  if (r.rest_counts) f -= rest.sum > 0.f ? (float)q_rest / rest.sum : 0.f;
  r.rest_f = r.coef * f;
  return r;
}
// One wave: the row's divergence (every lane has it).  Its terms are far larger than their sum
// where the student is near the teacher: fp64.
__device__ __forceinline__ float row_kl(const EntryLds &e, const RowCoefs &r, Softmax rest, double teacher_rest,
                                        const DistillParams &p) {
  const double shift = log(r.sum) - log(r.teacher_sum);
  double kl = 0;
  for (int j = threadIdx.x & 63; j < p.entries; j += 64) {
    if (e.token[j] == kNone) continue;
    const double q = power(e.t[j], r.teacher_ref, p) * r.teacher_f;
    if (q != 0) kl += q * (((e.t[j] - r.teacher_ref) - ((double)e.z[j] - r.ref)) * p.inv_temp + shift);
  }
  kl = wave_sum(kl);
  if (r.rest_counts) {
    const double q = power(teacher_rest, r.teacher_ref, p) * r.teacher_f;
    kl += q * (((teacher_rest - r.teacher_ref) - ((double)rest.ref - r.ref)) * p.inv_temp + shift - log((double)rest.sum));
  }
  return (float)kl;
}
// The gradient of entry j's token: the entries of one token write the same value.
__device__ __forceinline__ float entry_gradient(const EntryLds &e, int j, bool twice, const RowCoefs &r,
                                                const DistillParams &p) {
  const int token = e.token[j];
  double q = 0;
  if (twice) {
    for (int i = 0; i < p.entries; ++i)
      if (e.token[i] == token) q += power(e.t[i], r.teacher_ref, p);
  } else {
    q = power(e.t[j], r.teacher_ref, p);
  }
  return (float)(r.coef * (power(e.z[j], r.named_ref, p) * r.named_f - q * r.teacher_f));
}
// A vector of the rest's gradient.
template <class T, bool NT>
__device__ __forceinline__ void rest_gradient(T *dz, u32x4 v, float f, float ref, float k) {
  constexpr int N = Vec<T>::N;
  float x[N];
  Vec<T>::unpack(v, x);
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = f * pow2(x[e], k, ref);
  Vec<T>::template store<NT>(dz, x);
}
// The gradients of a row's named tokens, over what stands in their places.  Entry j's is computed by thread j, and
// stored by the wave that has stored its vector: a wave's stores to one address stay in their order.  (Vectors with
// holes and named tokens' elements in them afterwards are twice as many stores of parts of lines, which are slow where
// they go past the L2s: 4096 rows of 128256 bf16, 64 entries, 438 us, and 466 us with holes.)
// owner: of a vector (the row's last elements are that of one more).  Every thread calls it.
template <class T, int THR, class OWNER>
__device__ __forceinline__ void named_gradients(T *dz, const EntryLds &e, bool twice, const RowCoefs &coefs,
                                                const DistillParams &p, OWNER owner) {
  if ((int)threadIdx.x < p.entries) {
    const RowCoefs r = coefs;
    // (an entry's gradient takes all teacher's logits of its token: it has a place of its own)
    for (int j = threadIdx.x; j < p.entries; j += THR)
      if (e.token[j] != kNone) e.g[j] = entry_gradient(e, j, twice, r, p);
  }
  lds_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int j = threadIdx.x & 63; j < p.entries; j += 64) {
    const int token = e.token[j];
    if (token != kNone && owner(token / Vec<T>::N) == (int)threadIdx.x >> 6) Vec<T>::store1(dz + token, e.g[j]);
  }
}

enum { kForward = 0, kGradient = 1, kGradientNT = 2 };

// A row's marks: a byte for each held vector, K a thread side by side, so that a thread has its own
// with one load; then the other vectors' bits, in order; then a byte for each of the row's last V % N
// elements.  Where those start, and how many bytes all take (2^20 logits: 155 KB with the entries).
__host__ __device__ constexpr int tail_marks_of(int64_t vecs, int n, int held) {
  return held + (int)(((vecs > held ? vecs - held : 0) * n + 7) / 8);
}
__host__ __device__ constexpr size_t row_mark_bytes(int64_t vecs, int n, int held) {
  return ((size_t)tail_marks_of(vecs, n, held) + 8 + 15) / 16 * 16;
}
// The largest launch fits a CU's LDS: rows of the most tokens in fp32, held by 1024 threads with 16 vectors each or not
// held at all, with the most entries.
constexpr size_t largest_lds(int held) {
  return entry_lds_bytes(row_mark_bytes(HIMUON_TOP_VOCAB / Vec<float>::N, Vec<float>::N, held), HIMUON_TOP_MOST) +
         sizeof(EntrySums) + 16 * (sizeof(RowCoefs) + sizeof(Softmax));
}
static_assert(largest_lds(0) <= 160 << 10 && largest_lds(1024 * 16) <= 160 << 10, "LDS of the largest rows");
template <class T, int HELD>
__device__ __forceinline__ unsigned long_marks(const unsigned char *marks, int vec) {
  const int bit = (vec - HELD) * Vec<T>::N;
  return Vec<T>::N == 8 ? marks[HELD + (bit >> 3)] : marks[HELD + (bit >> 3)] >> (bit & 7) & 15u;
}

// One block per row: K vectors of 16 bytes a thread are held in registers between the softmax and
// the gradient, and where the row is LONG the vectors behind them are read again for the gradient.
// A forward pass over a LONG row holds none.
template <typename T, int THR, int K, bool LONG, int OUT>
__global__ __launch_bounds__(THR) void distill_row_kernel(const T *logits, T *dlogits, DistillParams p) {
  constexpr int N = Vec<T>::N, HELD = THR * K;
  constexpr bool GRAD = OUT != kForward, NT = OUT == kGradientNT;
  extern __shared__ u32x4 lds[];
  __shared__ EntrySums sums;
  __shared__ RowCoefs coefs[THR / 64];
  __shared__ Softmax parts[THR / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, V = p.vocab, vecs = V / N, tail_at = vecs * N + tid;
  const size_t mark_bytes = row_mark_bytes(LONG ? vecs : 0, N, HELD);
  const int tail_marks = tail_marks_of(LONG ? vecs : 0, N, HELD);
  const T *z = logits + row * p.ld_logits;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const EntryLds e = entry_lds(lds, mark_bytes, p.entries);
  const float w = gmem(p.weight)[row];
  int64_t token = kNone;   // of the thread's first entry
  float value = 0.f;
  if (tid < p.entries) {
    token = gmem(p.index)[row * p.ld_top + tid];
    value = entry_value(p, row * p.ld_top + tid);
  }
  const double teacher_rest = p.rest ? gmem(p.rest)[row] * p.temp : -__builtin_inf();
  for (int i = tid; i < (int)(mark_bytes / 16); i += THR) lds[i] = u32x4{0, 0, 0, 0};
  if (tid == 0) sums.named_max = sums.teacher_max = sums.twice = 0;
  if (w == 0.f) {
    if (tid == 0) gmem(p.kl)[row] = 0.f;
    if constexpr (GRAD) zero_row<T, THR, NT>(dz, V);
    return;
  }
  bool counts = token >= 0 && token < V;
  float student = counts ? Vec<T>::load1(z + token) : 0.f;
  u32x4 v[K > 0 ? K : 1];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    v[i] = u32x4{Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest};
    if (LONG || tid + i * THR < vecs) v[i] = Vec<T>::load(z + (tid + i * THR) * N);
  }
  float tail = tail_at < V ? Vec<T>::load1(z + tail_at) : -__builtin_inff();
  lds_barrier();

  // the entries: what they name is marked, their largest logits are found
  const int wave = tid >> 6, waves = (p.entries < THR ? p.entries + 63 : THR) >> 6;
  if (wave < waves) {
    unsigned top[2] = {0, 0};
    for (int j = tid; j < p.entries; j += THR) {
      if (j != tid) {
        token = gmem(p.index)[row * p.ld_top + j];
        value = entry_value(p, row * p.ld_top + j);
        counts = token >= 0 && token < V;
        student = counts ? Vec<T>::load1(z + token) : 0.f;
      }
      e.token[j] = counts ? (int)token : kNone;
      if (!counts) continue;
      e.t[j] = value;
      e.z[j] = student;
      top[0] = max(top[0], ordered(student));
      top[1] = max(top[1], ordered(value));
      const int vec = (int)token / N;
      if (vec == vecs) mark(e.marks, tail_marks + (int)token % N, 0, sums);
      else if (vec < HELD) mark(e.marks, vec % THR * K + vec / THR, (int)token % N, sums);
      else mark(e.marks, HELD + (((int)token - HELD * N) >> 3), ((int)token - HELD * N) & 7, sums);
    }
    top[0] = wave_max(top[0]);
    top[1] = wave_max(top[1]);
    if ((tid & 63) == 0) {
      atomicMax(&sums.named_max, top[0]);
      atomicMax(&sums.teacher_max, top[1]);
    }
  }
  lds_barrier();
  const bool twice = sums.twice != 0;
  if (wave < waves) {
    const float named_ref = ordered_ref(sums.named_max);
    const double teacher_ref = teacher_ref_of(sums.teacher_max, teacher_rest);
    double named = 0, teacher = tid == 0 ? power(teacher_rest, teacher_ref, p) : 0;
    for (int j = tid; j < p.entries; j += THR) {
      if (e.token[j] == kNone) continue;
      teacher += power(e.t[j], teacher_ref, p);
      if (first_of_token(e, j, twice)) named += power(e.z[j], named_ref, p);
    }
    named = wave_sum(named);
    teacher = wave_sum(teacher);
    if ((tid & 63) == 0) {
      sums.named[wave] = named;
      sums.teacher[wave] = teacher;
    }
  }
  unsigned char marks[K > 0 ? K : 1] = {};
  if constexpr (K > 0) __builtin_memcpy(marks, __builtin_assume_aligned(e.marks + tid * K, K), K);
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (marks[i]) hide<T>(v[i], marks[i]);
  if (tail_at < V && e.marks[tail_marks + tid]) tail = -__builtin_inff();

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
  int at = tid + HELD;
  if constexpr (LONG) {
    for (; at < vecs; at += THR) {
      u32x4 x = Vec<T>::load(z + (int64_t)at * N);
      const unsigned b = long_marks<T, HELD>(e.marks, at);
      if (b) hide<T>(x, b);
      m = max_of<T>(x, m);
      const float to = ref_of(m);
      sum = (sum > 0.f ? sum * pow2(ref, p.k, to) : sum) + sum_of<T>(x, p.k, to);
      ref = to;
    }
  }
  const Softmax rest = rest_join<THR / 64>(m, sum, p.k, parts);
  // (in LDS for later: the registers are full of the row)
  float rest_f, rest_ref;
  bool live;
  {
    const RowCoefs r = row_coefs(rest, sums, waves, teacher_rest, w, p);
    if ((tid & 63) == 0 && (wave < waves || wave == THR / 64 - 1)) coefs[wave] = r;
    rest_f = uniform(r.rest_f);
    rest_ref = uniform(r.rest_ref);
    live = r.live;
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (!live) {
    if (tid == 0) gmem(p.kl)[row] = 0.f;
    if constexpr (GRAD) zero_row<T, THR, NT>(dz, V);
    return;
  }
  if constexpr (GRAD) {
    if constexpr (LONG) {
      for (at -= THR; at >= HELD; at -= THR) {
        u32x4 x = Vec<T>::load(z + (int64_t)at * N);
        rest_gradient<T, NT>(dz + (int64_t)at * N, x, rest_f, rest_ref, p.k);
      }
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int vec = tid + i * THR;
      if (LONG || vec < vecs) rest_gradient<T, NT>(dz + vec * N, v[i], rest_f, rest_ref, p.k);
    }
    if (tail_at < V) Vec<T>::store1(dz + tail_at, rest_f * pow2(tail, p.k, rest_ref));
    named_gradients<T, THR>(dz, e, twice, coefs[wave], p, [&](int vec) { return vec == vecs ? 0 : vec % THR / 64; });
  }
  if (wave == THR / 64 - 1) {   // (the last wave: it has the fewest entries)
    const float kl = row_kl(e, coefs[wave], rest, teacher_rest, p);
    if ((tid & 63) == 0) gmem(p.kl)[row] = kl;
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

// A span's vectors and the row's last V % N elements, without the named ones; their marks are K bytes
// a thread, and a byte for each of the last elements.
template <typename T>
struct Span {
  static constexpr int N = Vec<T>::N, THR = kSpanThreads, K = kSpanK, kMarkBytes = kSpanVecs + 16;
  int v0, vecs, first, end, tail_at;   // of the row's vectors and elements
  bool has_tail;
  u32x4 v[K];
  float tail;
  unsigned char marks[K];

  __device__ __forceinline__ Span(const T *z, int V, int spans) {
    const int tid = threadIdx.x;
    v0 = blockIdx.x * kSpanVecs;
    vecs = V / N;
    first = v0 * N;
    end = (int)blockIdx.x == spans - 1 ? V : first + kSpanVecs * N;
    tail_at = vecs * N + tid;
    has_tail = (int)blockIdx.x == spans - 1 && tail_at < V;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int at = v0 + tid + i * THR;
      v[i] = u32x4{Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest};
      if (at < vecs) v[i] = Vec<T>::load(z + (int64_t)at * N);
    }
    tail = has_tail ? Vec<T>::load1(z + tail_at) : -__builtin_inff();
  }
  static __device__ __forceinline__ void clear(u32x4 *lds, EntrySums &sums) {
    if ((int)threadIdx.x < kMarkBytes / 16) lds[threadIdx.x] = u32x4{0, 0, 0, 0};
    if (threadIdx.x == 0) sums.named_max = sums.teacher_max = sums.twice = 0;
  }
  __device__ __forceinline__ bool holds(int64_t token) const { return token >= first && token < end; }
  __device__ __forceinline__ void mark_token(const EntryLds &e, int token, EntrySums &sums) const {
    const int vec = token / N - v0;
    if (vec + v0 == vecs) mark(e.marks, kSpanVecs + token % N, 0, sums);
    else mark(e.marks, vec % THR * K + vec / THR, token % N, sums);
  }
  __device__ __forceinline__ void hide_named(const EntryLds &e) {
    __builtin_memcpy(marks, __builtin_assume_aligned(e.marks + threadIdx.x * K, K), K);
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (marks[i]) hide<T>(v[i], marks[i]);
    if (has_tail && e.marks[kSpanVecs + threadIdx.x]) tail = -__builtin_inff();
  }
};

template <typename T>
__global__ __launch_bounds__(kSpanThreads) void distill_span_kernel(const T *logits, DistillParams p) {
  constexpr int THR = kSpanThreads;
  extern __shared__ u32x4 lds[];
  __shared__ EntrySums sums;
  __shared__ Softmax parts[THR / 64];
  const int64_t row = blockIdx.y;
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && row == 0 && tid == 0) *p.ticket = 0;
  if (gmem(p.weight)[row] == 0.f) return;
  const T *z = logits + row * p.ld_logits;
  const EntryLds e = entry_lds(lds, Span<T>::kMarkBytes, p.entries);
  Span<T>::clear(lds, sums);
  Span<T> s(z, p.vocab, gridDim.x);
  lds_barrier();
  for (int j = tid; j < p.entries; j += THR) {
    const int64_t token = gmem(p.index)[row * p.ld_top + j];
    e.token[j] = s.holds(token) ? (int)token : kNone;
    if (s.holds(token)) s.mark_token(e, (int)token, sums);
  }
  lds_barrier();
  const bool twice = sums.twice != 0;
  for (int j = tid; j < p.entries; j += THR)
    if (e.token[j] != kNone)
      gmem(p.entry)[row * p.entries + j] = f32x2{Vec<T>::load1(z + e.token[j]), first_of_token(e, j, twice) ? 1.f : 0.f};
  s.hide_named(e);
  float m = s.tail;
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) m = max_of<T>(s.v[i], m);
  const float ref = ref_of(m);
  float sum = pow2(s.tail, p.k, ref);
#pragma unroll
  for (int i = 0; i < kSpanK; ++i) sum += sum_of<T>(s.v[i], p.k, ref);
  const Softmax rest = rest_join<THR / 64>(m, sum, p.k, parts);
  if (tid == 0) gmem(p.spans)[row * gridDim.x + blockIdx.x] = f32x2{rest.ref, rest.sum};
}

// (without a gradient the grid has a row's first block alone)
template <typename T, bool GRAD>
__global__ __launch_bounds__(kSpanThreads) void distill_span_finish_kernel(const T *logits, T *dlogits, DistillParams p,
                                                                           int32_t spans, float *loss) {
  constexpr int THR = kSpanThreads, N = Vec<T>::N;
  extern __shared__ u32x4 lds[];
  __shared__ EntrySums sums;
  __shared__ RowCoefs coefs;
  __shared__ bool joins;
  const int64_t row = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63;
  T *dz = GRAD ? dlogits + row * p.ld_dlogits : nullptr;
  const EntryLds e = entry_lds(lds, Span<T>::kMarkBytes, p.entries);
  const float w = gmem(p.weight)[row];
  float kl = 0.f;
  if (w != 0.f || GRAD) {
    Span<T>::clear(lds, sums);
    Span<T> s(logits + row * p.ld_logits, GRAD && w != 0.f ? p.vocab : 0, GRAD ? spans : 0);
    RowCoefs r;
    r.live = false;
    if (w != 0.f) {
      const double teacher_rest = p.rest ? gmem(p.rest)[row] * p.temp : -__builtin_inf();
      lds_barrier();
      unsigned top[2] = {0, 0};
      for (int j = tid; j < p.entries; j += THR) {
        const int64_t token = gmem(p.index)[row * p.ld_top + j];
        const bool counts = token >= 0 && token < p.vocab;
        e.token[j] = counts ? (int)token : kNone;
        if (!counts) continue;
        const f32x2 x = gmem(p.entry)[row * p.entries + j];
        e.t[j] = entry_value(p, row * p.ld_top + j);
        e.z[j] = x[0];
        top[0] = max(top[0], ordered(x[0]));
        top[1] = max(top[1], ordered(e.t[j]));
        if (x[1] == 0.f) sums.twice = 1;
      }
      top[0] = wave_max(top[0]);
      top[1] = wave_max(top[1]);
      if (lane == 0) {
        atomicMax(&sums.named_max, top[0]);
        atomicMax(&sums.teacher_max, top[1]);
      }
      Softmax rest = {-__builtin_inff(), 0.f};
      for (int i = lane; i < spans; i += 64) {
        const f32x2 x = gmem(p.spans)[row * spans + i];
        const float m = __builtin_fmaxf(rest.ref, x[0]), to = ref_of(m);
        rest.sum = rest.sum * pow2(rest.ref, p.k, to) + x[1] * pow2(x[0], p.k, to);
        rest.ref = m;
      }
      const float m = wave_max(rest.ref);
      rest.sum = wave_sum(rest.sum * pow2(rest.ref, p.k, ref_of(m)));
      rest.ref = m;
      lds_barrier();
      const float named_ref = ordered_ref(sums.named_max);
      const double teacher_ref = teacher_ref_of(sums.teacher_max, teacher_rest);
      const bool twice = sums.twice != 0;
      double named = 0, teacher = tid == 0 ? power(teacher_rest, teacher_ref, p) : 0;
      for (int j = tid; j < p.entries; j += THR) {
        if (e.token[j] == kNone) continue;
        teacher += power(e.t[j], teacher_ref, p);
        if (first_of_token(e, j, twice)) named += power(e.z[j], named_ref, p);
      }
      named = wave_sum(named);
      teacher = wave_sum(teacher);
      if (lane == 0) {
        sums.named[tid >> 6] = named;
        sums.teacher[tid >> 6] = teacher;
      }
      lds_barrier();
      r = row_coefs(rest, sums, THR / 64, teacher_rest, w, p);
      if (r.live && blockIdx.x == 0 && tid < 64) kl = row_kl(e, r, rest, teacher_rest, p);
    }
    if constexpr (GRAD) {
      // (the span's own vectors were not read where the row is left out: its bounds are those of the call)
      const int v0 = blockIdx.x * kSpanVecs, vecs = p.vocab / N, tail_at = vecs * N + tid;
      const bool has_last = (int)blockIdx.x == spans - 1, has_tail = has_last && tail_at < p.vocab;
      if (!r.live) {
        const float zero[N] = {};
#pragma unroll
        for (int i = 0; i < kSpanK; ++i) {
          const int at = v0 + tid + i * THR;
          if (at < vecs) Vec<T>::template store<false>(dz + (int64_t)at * N, zero);
        }
        if (has_tail) Vec<T>::store1(dz + tail_at, 0.f);
      } else {
        const bool twice = sums.twice != 0;
#pragma unroll
        for (int i = 0; i < kSpanK; ++i) {
          const int at = v0 + tid + i * THR;
          if (at < vecs) rest_gradient<T, false>(dz + (int64_t)at * N, s.v[i], r.rest_f, r.rest_ref, p.k);
        }
        if (has_tail) Vec<T>::store1(dz + tail_at, r.rest_f * pow2(s.tail, p.k, r.rest_ref));
        if (tid == 0) coefs = r;
        lds_barrier();
        named_gradients<T, THR>(dz, e, twice, coefs, p, [&](int vec) {
          return vec == vecs ? (has_last ? 0 : -1) : vec < v0 || vec >= v0 + kSpanVecs ? -1 : (vec - v0) % THR / 64;
        });
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

// Whether rows are cut into spans.  Gradient in spans and by rows, us: 8 x 32000 bf16 12.4 and 11.4, 1 x 128256 11.3
// and 21.7, 32 x 128256 17.0 and 23.3, 128 x 128256 55.5 and 24.8, 32 x 262144 22.3 and 40.0, 100 x 262144 59.4 and 44.0,
// 8 x 50257 fp32 11.8 and 13.9.  Forward alone: 32 x 128256 11.0 and 16.4, 128 x 128256 17.6 and 18.0, 128 x 50257 fp32
// 14.3 and 12.6.
constexpr int kFewRows = 32, kFewRowsForward = 64, kFewVecs = 8192;
bool few_rows(const himuon_distill &p) {
  const int64_t vecs = p.vocab / (p.dtype == HIMUON_BF16 ? 8 : 4);
  return p.rows > 0 && vecs > kFewVecs && p.rows <= (p.dlogits ? kFewRows : kFewRowsForward);
}

// A gradient that the L2s together (32 MB) cannot hold goes past them (4096 x 128256 bf16 without left-out rows 503 us,
// 530 through them; 1000 x 50257 fp32 84 and 102; below that no difference).
constexpr double kL2Bytes = 32e6;

template <typename T, int THR, int K, bool LONG, int OUT>
void launch_rows(const T *z, T *dz, unsigned rows, const DistillParams &p, hipStream_t stream) {
  const size_t marks = row_mark_bytes(LONG ? p.vocab / Vec<T>::N : 0, Vec<T>::N, THR * K);
  hipLaunchKernelGGL((distill_row_kernel<T, THR, K, LONG, OUT>), dim3(rows), dim3(THR), entry_lds_bytes(marks, p.entries),
                     stream, z, dz, p);
}
template <typename T, int THR, int K, bool LONG = false>
void launch_rows(const T *z, T *dz, unsigned rows, int out, const DistillParams &p, hipStream_t stream) {
  if (out == kForward) launch_rows<T, THR, LONG ? 0 : K, LONG, kForward>(z, dz, rows, p, stream);
  else if (out == kGradient) launch_rows<T, THR, K, LONG, kGradient>(z, dz, rows, p, stream);
  else launch_rows<T, THR, K, LONG, kGradientNT>(z, dz, rows, p, stream);
}

template <typename T>
hipError_t launch_distill_t(const himuon_distill &c, const DistillParams &p, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  T *dz = reinterpret_cast<T *>(c.dlogits);
  const int64_t vecs = c.vocab / Vec<T>::N;
  if (few_rows(c)) {
    const unsigned spans = (unsigned)span_count(vecs), rows = (unsigned)c.rows;
    const size_t lds = entry_lds_bytes(Span<T>::kMarkBytes, c.k);
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
  return few_rows(p) ? 16 + (size_t)p.rows * (span_count(vecs) * sizeof(f32x2) + p.k * sizeof(f32x2)) : 0;
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
  p.spans = reinterpret_cast<f32x2 *>(reinterpret_cast<char *>(workspace) + 16);
  p.entry = reinterpret_cast<f32x2 *>(p.spans + c.rows * span_count(vecs));
  p.ld_logits = c.ld_logits;
  p.ld_dlogits = c.ld_dlogits;
  p.ld_top = c.ld_top;
  p.vocab = (int32_t)c.vocab;
  p.entries = c.k;
  p.value_bf16 = c.value_dtype == HIMUON_BF16;
  p.k = (float)(kLog2e / c.temperature);
  p.fine_k = kLog2e / c.temperature;
  p.temp = c.temperature;
  p.inv_temp = 1.0 / c.temperature;
  p.coef = (float)(c.grad_scale / c.temperature);
  return c.dtype == HIMUON_BF16 ? launch_distill_t<__bf16>(c, p, stream) : launch_distill_t<float>(c, p, stream);
}

}  // namespace himuon
