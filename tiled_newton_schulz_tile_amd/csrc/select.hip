// Choosing tokens from rows of logits: sampling with temperature, top-k, top-p and min-p from given
// random numbers (himuon_sample), and a row's k largest logits with the log-sum-exp of the others
// (himuon_top_logits).
//
// The order of a row's tokens is from the largest logit to the smallest, and among equal ones by
// index: a token's rank key is a 64-bit number, its logit's bits mapped to grow downwards above its
// index, unlike any other of the row.  Every filter keeps a first part of that order, so it is held
// as the last rank key that it keeps (its border).  A border is found by a descent over the digits
// of the rank key: a histogram of the elements in the present range, the bin in which the count (or
// the probability) reaches its target, and that bin as the next range, until one element is left.
//
// A block holds its row in registers (up to 256 KB; longer ones are read again for every pass).  What
// the filters may keep is most often a small part of the row: a bound on the smallest such logit is
// found first, the elements above it go into lists in LDS, and borders and draw come from those; rows
// whose lists overflow (flat ones) are read again.
//
// A border and a draw decide about whole tokens, and a sum in fp32 that is off by 1e-7 decides
// wrongly in one row of a hundred where 1e5 tokens share the probability.  Where a token hangs on
// them, powers are therefore taken in fp64 (fp64 multiply-adds run at the rate of fp32 ones here),
// sums of probabilities that go through atomics are whole multiples of a power of two in 64 bits, and
// all others have a fixed order: results do not depend on timing.
#include "device_common.h"
#include "himuon_internal.h"
#include "row_softmax.h"

#include <type_traits>

namespace himuon {
namespace {

typedef unsigned long long u64;

// The bits of a logit as a number that grows from the largest to the smallest (-0 as 0; any NaN
// before +inf).
__device__ __forceinline__ unsigned down_key(float z) {
  const unsigned u = __builtin_bit_cast(unsigned, z != z ? __builtin_nanf("") : z + 0.f);
  return u ^ ((unsigned)((int)~u >> 31) >> 1);
}
__device__ __forceinline__ u64 rank_key(float z, int index) { return (u64)down_key(z) << 32 | (unsigned)index; }

__device__ __forceinline__ float logit_of(unsigned down) {
  return __builtin_bit_cast(float, down & 0x80000000u ? down : down ^ 0x7fffffffu);
}
__device__ __forceinline__ float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }   // NaN wins

// Vector `vec` of a row of V elements; -inf stands in for what lies beyond the row.
template <class T>
__device__ __forceinline__ u32x4 row_vector(const T *z, int vec, int V) {
  constexpr int N = Vec<T>::N;
  u32x4 v = {Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest};
  if ((vec + 1) * N <= V) return Vec<T>::load(z + (int64_t)vec * N);
  if (vec * N >= V) return v;
  float x[N];
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = vec * N + e < V ? Vec<T>::load1(z + vec * N + e) : -__builtin_inff();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (N == 8) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);   // (exact)
    else v[i] = __builtin_bit_cast(unsigned, x[i]);
  }
  return v;
}

// Where elements come from: each(f) calls f(index, logit) for all of them, the threads of the block
// in step.  A row in memory:
template <class T, int THR>
struct RowSource {
  const T *z;
  int V;
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    constexpr int N = Vec<T>::N;
    for (int at = threadIdx.x; at * N < V; at += THR) {
      float x[N];
      Vec<T>::unpack(row_vector(z, at, V), x);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (at * N + e < V) f(at * N + e, x[e]);
    }
  }
};
// A row in registers: K vectors a thread.  Each wave has a stretch of 64 K consecutive vectors, so
// that elements are in order from wave to wave.
template <class T, int K>
struct HeldRow {
  u32x4 v[K];
  int first, V;   // the thread's first vector

  __device__ __forceinline__ HeldRow(const T *z, int vocab) {
    first = (threadIdx.x >> 6) * 64 * K + (threadIdx.x & 63);
    V = vocab;
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = row_vector(z, first + 64 * i, V);
  }
  // f(index of the vector's first element, its elements), one vector after the other: the compiler
  // may neither keep the unpacked elements of one sweep for the next nor mix the vectors of a sweep
  // (both would take far more registers than there are).
  template <class F>
  __device__ __forceinline__ void vectors(F f) {
    constexpr int N = Vec<T>::N;
    int at = first;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      asm volatile("" : "+v"(v[i]), "+v"(at));
      float x[N];
      Vec<T>::unpack(v[i], x);
      f((at + 64 * i) * N, x);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};
// Rank keys in LDS: a list for each wave, in the order of their indices.
constexpr int kListMost = 512;
struct ListSource {
  const u64 *list;   // of this thread's wave
  int n;
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int j = threadIdx.x & 63; j < n; j += 64) {
      const u64 r = list[j];
      f((int)(unsigned)r, logit_of((unsigned)(r >> 32)));
    }
  }
};
// One logit a thread.
struct ThreadSource {
  float z;
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    f((int)threadIdx.x, z);
  }
};

// Appends a vector's elements from `least` on to the wave's list of n keys (of which kListMost are
// kept; n counts on).
// Whether the wave has any.
template <int N>
__device__ __forceinline__ bool append(u64 *list, int &n, int at, const float (&x)[N], float least, int V) {
  float top = x[0];
#pragma unroll
  for (int e = 1; e < N; ++e) top = maximum(top, x[e]);
  if (!__any(top >= least)) return false;
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (x[e] >= least && at + e < V) m |= 1u << e;
  const int count = __builtin_popcount(m);
  int pos = n;
#pragma unroll
  for (int b = 0; 1 << b <= N; ++b) {
    const u64 with = __ballot(count >> b & 1);
    pos += __builtin_amdgcn_mbcnt_hi((unsigned)(with >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)with, 0)) << b;
    n += __builtin_popcountll(with) << b;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (m >> e & 1) {
      if (pos < kListMost) list[pos] = rank_key(x[e], at + e);
      ++pos;
    }
  return true;
}

constexpr int kBins = 1024;
struct SelectLds {
  u64 mass[kBins];      // what a bin weighs
  unsigned count[kBins];
  u64 wave[16];
  u64 before;           // the weight before the bin that was found
  int bin;
};

template <int THR>
__device__ __forceinline__ u64 block_scan(u64 mine, u64 *wave, u64 &total) {   // exclusive
  const int lane = threadIdx.x & 63;
  u64 s = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const u64 up = __shfl_up(s, d);
    if (lane >= d) s += up;
  }
  if (lane == 63) wave[threadIdx.x >> 6] = s;
  __syncthreads();
  u64 base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THR / 64; ++w) {
    if (w < (int)(threadIdx.x >> 6)) base += wave[w];
    total += wave[w];
  }
  __syncthreads();
  return base + s - mine;
}

// The last rank key, from first to last, up to which the elements weigh `target` at least: the first
// one that reaches it.  weight(z): an element's weight (all together below 2^64).  Where all weigh
// less: last.  target_of(total): the target, at least 1, given what all weigh together.  With LEVELS
// > 0 the descent ends after so many, at a key that is no smaller.
template <int THR, int LEVELS = 0, class SOURCE, class WEIGHT, class TARGET>
__device__ __forceinline__ u64 find_border(SOURCE &src, u64 first, u64 last, WEIGHT weight, TARGET target_of,
                                           SelectLds &lds) {
  constexpr int B = kBins / THR > 0 ? kBins / THR : 1;   // bins a thread
  u64 base = 0, target = 0;
  const u64 end = last;
  for (int level = 1;; ++level) {
    const int bits = 64 - __builtin_clzll((last - first) | 1);
    const int shift = bits > 10 ? bits - 10 : 0;
#pragma unroll
    for (int i = 0; i < kBins; i += THR)
      if (i + (int)threadIdx.x < kBins) {
        lds.mass[i + threadIdx.x] = 0;
        lds.count[i + threadIdx.x] = 0;
      }
    __syncthreads();
    src.each([&](int index, float z) {
      const u64 r = rank_key(z, index);
      if (r < first || r > last) return;
      const int bin = (int)((r - first) >> shift);
      const u64 w = weight(z);
      atomicAdd(&lds.count[bin], 1u);
      if (w) atomicAdd(&lds.mass[bin], w);
    });
    __syncthreads();
    u64 w[B], mine = 0, total;
#pragma unroll
    for (int i = 0; i < B; ++i) mine += w[i] = (int)threadIdx.x * B + i < kBins ? lds.mass[threadIdx.x * B + i] : 0;
    u64 before = base + block_scan<THR>(mine, lds.wave, total);
    if (level == 1) {
      target = target_of(total);
      if (total < target) return end;
    }
    if (before < target && before + mine >= target) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        if (before < target && before + w[i] >= target) {
          lds.bin = threadIdx.x * B + i;
          lds.before = before;
        }
        before += w[i];
      }
    }
    __syncthreads();
    base = lds.before;
    first += (u64)lds.bin << shift;
    last = last - first < ((u64)1 << shift) - 1 ? last : first + (((u64)1 << shift) - 1);
    const bool done = shift == 0 || lds.count[lds.bin] == 1 || level == LEVELS;
    __syncthreads();
    if (done) return last;
  }
}

struct SampleParams {
  const float *uniform;
  const float *temperature, *top_p, *min_p;   // nullptr: all rows alike, as below
  const int32_t *top_k;
  int64_t *token;
  float *logp, *kept;
  int64_t ld_logits;
  int32_t vocab;
  int32_t k;
  int32_t mass_bits;        // probabilities in histograms are multiples of 2^-mass_bits of the largest
  double T, p, m;
};

// What a row's settings come to.
struct Settings {
  double temp, k;   // k: log2(e) / temperature
  double top_p, min_p;
  int top_k;        // V: off
  bool greedy, good, by_k, by_p;
};
__device__ __forceinline__ Settings settings_of(const SampleParams &p, int64_t row) {
  Settings s;
  s.temp = p.temperature ? (double)gmem(p.temperature)[row] : p.T;
  s.top_p = p.top_p ? (double)gmem(p.top_p)[row] : p.p;
  s.min_p = p.min_p ? (double)gmem(p.min_p)[row] : p.m;
  s.top_k = p.top_k ? gmem(p.top_k)[row] : p.k;
  s.greedy = s.temp == 0.;
  s.good = s.greedy || (s.temp >= 0x1p-20 && s.temp <= 0x1p20);
  if (s.greedy) {   // the first token of all
    s.temp = s.top_k = 1;
    s.top_p = 1.;
    s.min_p = 0.;
  }
  if (!s.good) s.temp = 1.;
  s.k = kLog2e / s.temp;
  if (s.top_k <= 0 || s.top_k > p.vocab) s.top_k = p.vocab;
  s.top_p = s.top_p > 0. ? s.top_p : s.top_p <= 0. ? 0. : 1.;   // (NaN: off)
  s.min_p = s.min_p > 0. ? (s.min_p < 1. ? s.min_p : 1.) : 0.;
  s.by_k = s.top_k < p.vocab;
  s.by_p = s.top_p < 1.;
  return s;
}
// The place of a draw, as a share of what is kept.
__device__ __forceinline__ double uniform_of(const SampleParams &p, int64_t row) {
  const double u = (double)gmem(p.uniform)[row];
  return u > 0. ? (u < 1. ? u : 1.) : 0.;   // (NaN is 0)
}
__device__ __forceinline__ void write_bad(const SampleParams &p, int64_t row) {
  gmem(p.token)[row] = -1;
  gmem(p.logp)[row] = gmem(p.kept)[row] = __builtin_nanf("");
}
// top, all, kept: the largest logit, and the sums of powers of the distances to it.
__device__ __forceinline__ void write_token(const SampleParams &p, int64_t row, const Settings &s, int token, float logit,
                                            float top, double all, double kept) {
  gmem(p.token)[row] = token;
  gmem(p.logp)[row] = s.greedy ? 0.f : (float)(((double)logit - top) / s.temp - log(all));
  gmem(p.kept)[row] = s.greedy ? 1.f : (float)(kept / all);
}

// Powers of the distances to the row's largest logit, 2^-1010 at least: those below kNoPower are none.
constexpr double kNoPower = 0x1p-1000;
struct Powers {
  float top;
  double k, unit;   // unit: multiples of 1 / unit in histograms
  __device__ __forceinline__ double of(float z) const {
    const double magic = 0x1.8p52, d = __builtin_fmax((double)z - top, -1010. / k);
    const double a = __builtin_fma(d, k, magic), f = __builtin_fma(d, k, magic - a);
    const u64 p = __builtin_bit_cast(u64, pow2_fraction(f));
    // (the low bits of a are the exponent)
    return __builtin_bit_cast(double, p + (__builtin_bit_cast(u64, a) << 52));
  }
  __device__ __forceinline__ u64 mass(float z) const { return (u64)(of(z) * unit + 0.5); }
};
constexpr u64 kLastKey = (u64)0xff7fffffu << 32 | 0xffffffffu;   // of a finite logit

// What a row's filters keep, once their borders are known.
struct Kept {
  u64 border;       // the last rank key of top_k and top_p
  double least;     // the least power of min_p, kNoPower at least
  __device__ __forceinline__ double power(const Powers &e, int index, float z) const {
    const double x = e.of(z);
    return rank_key(z, index) <= border && x >= least ? x : 0.;
  }
};

// The borders of top_k and top_p together.  all: the sum of the row's powers where top_p needs it (it
// does not with top_k: then it is that of the first top_k).
template <int THR, class SOURCE>
__device__ __forceinline__ u64 filter_border(SOURCE &src, u64 first, u64 last, const Settings &s, const Powers &e, double all,
                                             SelectLds &lds) {
  u64 border = last;
  if (s.by_k)
    border = find_border<THR>(src, first, last, [](float) { return (u64)1; }, [&](u64) { return (u64)s.top_k; }, lds);
  if (s.by_p)
    border = find_border<THR>(src, first, border, [&](float z) { return e.mass(z); }, [&](u64 total) {
      const double t = __builtin_ceil(s.top_p * (s.by_k ? (double)total : all * e.unit));
      return t < 1. ? (u64)1 : (u64)t;
    }, lds);
  return border;
}

template <int THR>
__device__ __forceinline__ double block_sum_in_order(double x, double *wave) {
  x = wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int w = 0; w < THR / 64; ++w) s += wave[w];
  return s;
}
template <int THR>
__device__ __forceinline__ float block_maximum(float x, float *wave) {
  x = wave_reduce(x, -__builtin_inff(), [](float a, float b) { return maximum(a, b); });
  if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = x;
  __syncthreads();
  x = wave[0];
#pragma unroll
  for (int w = 1; w < THR / 64; ++w) x = maximum(x, wave[w]);
  return x;
}
__device__ __forceinline__ double wave_scan(double x) {   // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double up = __shfl_up(x, d);
    if (lane >= d) x += up;
  }
  return x;
}

// One wave: which of n parts (0 or more each, in order) the target falls into: the first one up to
// which they sum to more; the last that is not 0 if none does.  before: the sum before it.
template <class PART>
__device__ __forceinline__ int find_part(int n, double target, PART part, double &before) {
  const int lane = threadIdx.x & 63;
  double sum = 0;
  int last = 0;
  double last_before = 0;
  for (int c = 0; c < n; c += 64) {
    const double w = c + lane < n ? part(c + lane) : 0., s = wave_scan(w);
    const u64 hit = __ballot(w > 0. && sum + s > target), some = __ballot(w > 0.);
    if (hit || some) {
      const int l = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some);
      const double up = __shfl(s - w, l);
      last = c + l;
      last_before = sum + up;
      if (hit) break;
    }
    sum += __shfl(s, 63);
  }
  before = last_before;
  return last;
}

// The token of a row that is read from memory for every pass over it; chunk: LDS, one for each wave
// and turn over the row's vectors.
template <class T, int THR>
__device__ __forceinline__ void sample_from_memory(const T *z, float top, const Settings &s, const Powers &e, int64_t row,
                                                   const SampleParams &p, SelectLds &lds, double *wave, double *chunk) {
  constexpr int N = Vec<T>::N, W = THR / 64;
  const int tid = threadIdx.x, lane = tid & 63, V = p.vocab, vecs = (V + N - 1) / N;
  RowSource<T, THR> src = {z, V};
  double all = 0;
  src.each([&](int, float x) { all += e.of(x); });
  all = block_sum_in_order<THR>(all, wave);
  const Kept kept = {s.by_k || s.by_p ? filter_border<THR>(src, (u64)down_key(top) << 32, kLastKey, s, e, all, lds) : ~(u64)0,
                     __builtin_fmax(s.min_p, kNoPower)};
  const auto weigh = [&](int vec, float (&x)[N]) {
    Vec<T>::unpack(row_vector(z, vec, V), x);
    double t = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) t += kept.power(e, vec * N + i, x[i]);
    return t;
  };
  // the draw: a wave's 64 vectors of a turn are consecutive, so the chunks are in order
  const int turns = (vecs + THR - 1) / THR, chunks = turns * W;
  float x[N];
  for (int t = 0; t < turns; ++t) {
    const double sum = wave_sum(weigh(t * THR + tid, x));
    if (lane == 0) chunk[t * W + (tid >> 6)] = sum;
  }
  __syncthreads();
  if (tid >= 64) return;
  double total = 0;
  for (int c = lane; c < chunks; c += 64) total += chunk[c];
  total = wave_sum(total);
  const double target = uniform_of(p, row) * total;
  double before, more, last;
  const int c = find_part(chunks, target, [&](int i) { return chunk[i]; }, before);
  const double own = weigh(c * 64 + lane, x);
  const int v = c * 64 + find_part(64, target - before, [&](int) { return own; }, more);
  const int n = N < V - v * N ? N : V - v * N;
  const float mine = Vec<T>::load1(z + (lane < n ? v * N + lane : V - 1));
  const int i = find_part(n, target - before - more, [&](int j) { return kept.power(e, v * N + j, mine); }, last);
  if (lane == i) write_token(p, row, s, v * N + i, mine, top, all, total);
}

// A row that is held in registers, one block for it.
template <class T, int THR, int K>
__global__ __launch_bounds__(THR) void sample_kernel(const T *logits, SampleParams p) {
  constexpr int N = Vec<T>::N, W = THR / 64;
  static_assert(64 * K <= THR && K <= kListMost, "a wave's stretch is one vector a thread; its turns fit in its list");
  __shared__ SelectLds lds;
  __shared__ u64 lists[W][kListMost];
  __shared__ double wave[W];
  __shared__ float wave_top[W];
  __shared__ int counts[W];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, V = p.vocab;
  const T *z = logits + row * p.ld_logits;
  const Settings s = settings_of(p, row);
  HeldRow<T, K> held(z, V);
  float mine = -__builtin_inff();
  held.vectors([&](int, const float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) mine = maximum(mine, x[e]);
  });
  const float top = block_maximum<THR>(mine, wave_top);
  if (!(__builtin_fabsf(top) < __builtin_inff()) || !s.good) {   // NaN or +inf in the row, nothing but -inf, no such temperature
    if (tid == 0) write_bad(p, row);
    return;
  }
  const Powers e = {top, s.k, __builtin_amdgcn_ldexp(1., p.mass_bits)};
  double all = 0;
  if (s.by_k || s.by_p || s.min_p > 0.) {
    // a logit that the filters' last token is not below
    const u64 first = (u64)down_key(top) << 32;
    const auto below = [&](double b) {   // b, and errors of 1e-6
      return (float)__builtin_fmax(b - 1e-6 * (__builtin_fabs(b) + __builtin_fabs(top)), -__FLT_MAX__);
    };
    float least = -__FLT_MAX__;
    if (s.greedy) {
      least = top;
    } else if (s.by_k && s.top_k <= THR) {
      // that many threads' largest ones are not below their top_k-th
      ThreadSource src = {mine};
      const u64 b = find_border<THR, 2>(src, first, kLastKey, [](float) { return (u64)1; }, [&](u64) { return (u64)s.top_k; }, lds);
      least = logit_of((unsigned)(b >> 32));
    } else if (s.by_p && !s.by_k) {
      // all tokens below it have less than 1 - top_p of what the largest one alone has
      least = below(top + s.temp * log((1. - s.top_p) / V));
    }
    if (s.min_p > 0. && !(s.by_k && s.by_p)) least = __builtin_fmaxf(least, below(top + s.temp * log(s.min_p)));
    // (without a bound every element goes into the lists: only where they hold a row)
    int n = least > -__FLT_MAX__ || V <= W * kListMost ? 0 : kListMost + 1;
    if (n == 0) {
      if (s.by_p && !s.by_k) {
        held.vectors([&](int at, const float (&x)[N]) {
          append(lists[tid >> 6], n, at, x, least, V);
          double t = 0;
#pragma unroll
          for (int i = 0; i < N; ++i) t += e.of(x[i]);
          all += t;
        });
      } else {
        // the sum is not for a border: below the bound, powers are fp32 with the exponent's product in two parts
        const float hi = (float)s.k, lo = (float)(s.k - hi);
        held.vectors([&](int at, const float (&x)[N]) {
          float y[N];
#pragma unroll
          for (int i = 0; i < N; ++i) y[i] = x[i];
          if (append(lists[tid >> 6], n, at, x, least, V)) {
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = x[i] < least ? x[i] : -__builtin_inff();
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float d = __builtin_fmaxf(y[i] - top, -__FLT_MAX__);
            y[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(d, hi, d * lo));
          }
#pragma unroll
          for (int d = 1; d < N; d *= 2)
#pragma unroll
            for (int i = 0; i < N; i += 2 * d) y[i] += y[i + d];
          all += (double)y[0];
        });
      }
    }
    ListSource src = {lists[tid >> 6], n <= kListMost ? n : 0};
    if (!(s.by_p && !s.by_k)) src.each([&](int, float x) { all += e.of(x); });
    if (lane == 0) counts[tid >> 6] = n;
    all = block_sum_in_order<THR>(all, wave);
    bool fits = true;
#pragma unroll
    for (int w = 0; w < W; ++w) fits = fits && counts[w] <= kListMost;
    if (!fits) {
      __syncthreads();
      sample_from_memory<T, THR>(z, top, s, e, row, p, lds, wave, reinterpret_cast<double *>(&lists[0][0]));
      return;
    }
    const Kept kept = {s.by_k || s.by_p ? filter_border<THR>(src, first, kLastKey, s, e, all, lds) : ~(u64)0,
                       __builtin_fmax(s.min_p, kNoPower)};
    // the draw, over the lists in the order of their indices
    double t = 0;
    src.each([&](int index, float x) { t += kept.power(e, index, x); });
    const double total = block_sum_in_order<THR>(t, wave), target = uniform_of(p, row) * total;
    if (tid >= 64) return;
    double before, more;
    const int w = find_part(W, target, [&](int i) { return wave[i]; }, before);
    const u64 *list = lists[w];
    const auto at = [&](int j) { return kept.power(e, (int)(unsigned)list[j], logit_of((unsigned)(list[j] >> 32))); };
    const int j = find_part(counts[w], target - before, at, more);
    if (lane == 0) write_token(p, row, s, (int)(unsigned)list[j], logit_of((unsigned)(list[j] >> 32)), top, all, total);
    return;
  }

  // all tokens: what each wave's stretch weighs, then the vectors of one stretch
  held.vectors([&](int, const float (&x)[N]) {
    double t = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) t += e.of(x[i]);
    all += t;
  });
  all = block_sum_in_order<THR>(all < 0x1p-980 ? 0. : all, wave);   // (nothing but powers that are none)
  const Kept kept = {~(u64)0, kNoPower};
  const double target = uniform_of(p, row) * all;
  double before;
  const int w = find_part(W, target, [&](int i) { return wave[i]; }, before);   // (every wave finds the same)
  float x[N];
  const int vec = w * 64 * K + tid;
  Vec<T>::unpack(row_vector(z, tid < 64 * K ? vec : V, V), x);
  double t = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) t += kept.power(e, vec * N + i, x[i]);
  double *part = reinterpret_cast<double *>(&lists[0][0]);
  part[tid] = t;
  __syncthreads();
  if (tid >= 64) return;
  double more, last;
  const int v = w * 64 * K + find_part(64 * K, target - before, [&](int i) { return part[i]; }, more);
  const int n = N < V - v * N ? N : V - v * N;
  const float own = Vec<T>::load1(z + (lane < n ? v * N + lane : V - 1));
  const int i = find_part(n, target - before - more, [&](int j) { return kept.power(e, v * N + j, own); }, last);
  if (lane == i) write_token(p, row, s, v * N + i, own, top, all, all);
}

// A row that is too long for that.
template <class T, int THR>
__global__ __launch_bounds__(THR) void sample_long_kernel(const T *logits, SampleParams p) {
  extern __shared__ double chunk[];
  __shared__ SelectLds lds;
  __shared__ double wave[THR / 64];
  __shared__ float wave_top[THR / 64];
  const int64_t row = blockIdx.x;
  const T *z = logits + row * p.ld_logits;
  const RowSource<T, THR> src = {z, p.vocab};
  const Settings s = settings_of(p, row);
  float mine = -__builtin_inff();
  src.each([&](int, float x) { mine = maximum(mine, x); });
  const float top = block_maximum<THR>(mine, wave_top);
  if (!(__builtin_fabsf(top) < __builtin_inff()) || !s.good) {
    if (threadIdx.x == 0) write_bad(p, row);
    return;
  }
  const Powers e = {top, s.k, __builtin_amdgcn_ldexp(1., p.mass_bits)};
  sample_from_memory<T, THR>(z, top, s, e, row, p, lds, wave, chunk);
}

struct TopParams {
  void *value;
  int64_t *index;
  float *rest;
  int64_t ld_logits, ld_top;
  int32_t vocab, k;
  float k2;         // log2(e) / temperature
  float inv_temp;
};

// Sorts n keys (a power of two, 64 at least).
template <int THR>
__device__ __forceinline__ void sort_keys(u64 *keys, int n) {
  for (int size = 2; size <= n; size *= 2)
    for (int step = size / 2; step > 0; step /= 2) {
      for (int i = threadIdx.x; i < n / 2; i += THR) {
        const int a = 2 * i - (i & (step - 1)), b = a + step;
        const u64 x = keys[a], y = keys[b];
        if ((x > y) == !(a & size)) {
          keys[a] = y;
          keys[b] = x;
        }
      }
      __syncthreads();
    }
}
__device__ __forceinline__ int sort_size(int n) { return n <= 64 ? 64 : 1 << (32 - __builtin_clz(n - 1)); }

template <int THR>
struct TopLds {
  SelectLds select;
  u64 keys[HIMUON_TOP_MOST];   // the largest, to be sorted
  Softmax waves[THR / 64];
  int n;
};

// The elements of a source up to border (k of them) are sorted and written; the others' sum.
template <class T, int THR, class SOURCE>
__device__ __forceinline__ void write_top(SOURCE &src, u64 border, const TopParams &p, int64_t row, TopLds<THR> &lds) {
  const int n = sort_size(p.k);
  for (int i = threadIdx.x; i < n; i += THR) lds.keys[i] = ~(u64)0;
  if (threadIdx.x == 0) lds.n = 0;
  __syncthreads();
  src.each([&](int index, float x) {
    const u64 r = rank_key(x, index);
    if (r <= border) lds.keys[atomicAdd(&lds.n, 1)] = r;
  });
  __syncthreads();
  sort_keys<THR>(lds.keys, n);
  for (int i = threadIdx.x; i < p.k; i += THR) {
    const u64 r = lds.keys[i];
    gmem(p.index)[row * p.ld_top + i] = (int)(unsigned)r;
    Vec<T>::store1(reinterpret_cast<T *>(p.value) + row * p.ld_top + i, logit_of((unsigned)(r >> 32)));
  }
}
template <int THR>
__device__ __forceinline__ void write_rest(float max, float sum, const TopParams &p, int64_t row, TopLds<THR> &lds) {
  const Softmax s = block_softmax<THR / 64>(max, sum, p.k2, lds.waves);
  if (threadIdx.x == 0)
    gmem(p.rest)[row] = s.sum == 0.f ? -__builtin_inff() : s.ref * p.inv_temp + kLn2 * __builtin_amdgcn_logf(s.sum);
}
// The same from a whole row, by its border.
template <class T, int THR, class SOURCE>
__device__ __forceinline__ void top_of_all(SOURCE &src, const TopParams &p, int64_t row, TopLds<THR> &lds) {
  u64 border = ~(u64)0;
  if (p.k < p.vocab)
    border = find_border<THR>(src, 0, ~(u64)0, [](float) { return (u64)1; }, [&](u64) { return (u64)p.k; }, lds.select);
  write_top<T, THR>(src, border, p, row, lds);
  float m = -__builtin_inff(), sum = 0.f;
  src.each([&](int index, float x) {
    if (rank_key(x, index) > border) m = __builtin_fmaxf(m, x);
  });
  const float ref = ref_of(m);
  src.each([&](int index, float x) {
    if (rank_key(x, index) > border) sum += pow2(x, p.k2, ref);
  });
  write_rest<THR>(m, sum, p, row, lds);
}

template <class T, int THR, int K>
__global__ __launch_bounds__(THR) void top_kernel(const T *logits, TopParams p) {
  constexpr int N = Vec<T>::N, W = THR / 64;
  __shared__ TopLds<THR> lds;
  __shared__ u64 lists[W][kListMost];
  __shared__ float wave_top[W];
  __shared__ int counts[W];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, V = p.vocab;
  const T *z = logits + row * p.ld_logits;
  HeldRow<T, K> held(z, V);
  float mine = -__builtin_inff();
  held.vectors([&](int, const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) mine = maximum(mine, x[i]);
  });
  const float top = block_maximum<THR>(mine, wave_top);
  if (!(__builtin_fabsf(top) < __builtin_inff()) || p.k > THR) {
    RowSource<T, THR> src = {z, V};
    top_of_all<T, THR>(src, p, row, lds);
    return;
  }
  // that many threads' largest logits are not below their k-th; no border: fewer threads have any
  ThreadSource threads = {mine};
  const u64 bound = find_border<THR, 2>(threads, (u64)down_key(top) << 32, kLastKey, [](float) { return (u64)1; },
                                        [&](u64) { return (u64)p.k; }, lds.select);
  const float least = bound == kLastKey ? -__builtin_inff() : logit_of((unsigned)(bound >> 32));
  int n = 0;
  float sum = 0.f;
  const float ref = ref_of(least);
  held.vectors([&](int at, const float (&x)[N]) {
    float y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = x[i];
    if (append(lists[tid >> 6], n, at, x, least, V)) {
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = x[i] < least ? x[i] : -__builtin_inff();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = pow2(y[i], p.k2, ref);
#pragma unroll
    for (int d = 1; d < N; d *= 2)
#pragma unroll
      for (int i = 0; i < N; i += 2 * d) y[i] += y[i + d];
    sum += y[0];
  });
  if (lane == 0) counts[tid >> 6] = n;
  const float others = block_softmax<W>(sum > 0.f ? least : -__builtin_inff(), sum, p.k2, lds.waves).sum;
  bool fits = true;
#pragma unroll
  for (int w = 0; w < W; ++w) fits = fits && counts[w] <= kListMost;
  // (where the others are so far below that their powers lose bits, they are taken from their own largest)
  if (!fits || !(others >= 0x1p-60f || least == -__builtin_inff())) {
    __syncthreads();
    RowSource<T, THR> src = {z, V};
    top_of_all<T, THR>(src, p, row, lds);
    return;
  }
  ListSource src = {lists[tid >> 6], n};
  const u64 border = find_border<THR>(src, (u64)down_key(top) << 32, ~(u64)0, [](float) { return (u64)1; },
                                      [&](u64) { return (u64)p.k; }, lds.select);
  write_top<T, THR>(src, border, p, row, lds);
  float m = sum > 0.f ? least : -__builtin_inff();
  src.each([&](int index, float x) {
    if (rank_key(x, index) > border) m = __builtin_fmaxf(m, x);
  });
  const float to = ref_of(m);
  if (sum > 0.f) sum *= pow2(least, p.k2, to);
  src.each([&](int index, float x) {
    if (rank_key(x, index) > border) sum += pow2(x, p.k2, to);
  });
  write_rest<THR>(m, sum, p, row, lds);
}

template <class T, int THR>
__global__ __launch_bounds__(THR) void top_long_kernel(const T *logits, TopParams p) {
  __shared__ TopLds<THR> lds;
  RowSource<T, THR> src = {logits + blockIdx.x * p.ld_logits, p.vocab};
  top_of_all<T, THR>(src, p, blockIdx.x, lds);
}

constexpr int64_t kLaunchRows = (int64_t)1 << 21;   // a grid holds fewer than 2^32 threads

// A row's vectors by the block that holds them: f(kernel's threads, vectors a thread; 0: too long).
template <class F>
void with_shape(int64_t vecs, F f) {
  if (vecs <= 256) f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
  else if (vecs <= 256 * 4) f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
  else if (vecs <= 512 * 8) f(std::integral_constant<int, 512>(), std::integral_constant<int, 8>());
  else if (vecs <= 1024 * 8) f(std::integral_constant<int, 1024>(), std::integral_constant<int, 8>());
  else if (vecs <= 1024 * 16) f(std::integral_constant<int, 1024>(), std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 1024>(), std::integral_constant<int, 0>());
}

template <class T>
hipError_t launch_sample_t(const himuon_sampling &c, SampleParams p, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  const int64_t vecs = (c.vocab + Vec<T>::N - 1) / Vec<T>::N;
  for (int64_t r = 0; r < c.rows; r += kLaunchRows) {
    const unsigned rows = (unsigned)(c.rows - r < kLaunchRows ? c.rows - r : kLaunchRows);
    with_shape(vecs, [&](auto threads, auto held) {
      constexpr int THR = decltype(threads)::value, K = decltype(held)::value;
      const T *at = z + r * c.ld_logits;
      if constexpr (K > 0) {
        hipLaunchKernelGGL((sample_kernel<T, THR, K>), dim3(rows), dim3(THR), 0, stream, at, p);
      } else {
        const size_t lds = (vecs + THR - 1) / THR * (THR / 64) * sizeof(double);
        hipLaunchKernelGGL((sample_long_kernel<T, THR>), dim3(rows), dim3(THR), lds, stream, at, p);
      }
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.uniform += rows;
    if (p.temperature) p.temperature += rows;
    if (p.top_k) p.top_k += rows;
    if (p.top_p) p.top_p += rows;
    if (p.min_p) p.min_p += rows;
    p.token += rows;
    p.logp += rows;
    p.kept += rows;
  }
  return hipSuccess;
}

template <class T>
hipError_t launch_top_t(const himuon_top &c, TopParams p, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  const int64_t vecs = (c.vocab + Vec<T>::N - 1) / Vec<T>::N;
  for (int64_t r = 0; r < c.rows; r += kLaunchRows) {
    const unsigned rows = (unsigned)(c.rows - r < kLaunchRows ? c.rows - r : kLaunchRows);
    with_shape(vecs, [&](auto threads, auto held) {
      constexpr int THR = decltype(threads)::value, K = decltype(held)::value;
      const T *at = z + r * c.ld_logits;
      if constexpr (K > 0) hipLaunchKernelGGL((top_kernel<T, THR, K>), dim3(rows), dim3(THR), 0, stream, at, p);
      else hipLaunchKernelGGL((top_long_kernel<T, THR>), dim3(rows), dim3(THR), 0, stream, at, p);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.value = reinterpret_cast<T *>(p.value) + rows * p.ld_top;
    p.index += rows * p.ld_top;
    p.rest += rows;
  }
  return hipSuccess;
}

}  // namespace

size_t sample_workspace(const himuon_sampling &) { return 0; }
size_t top_workspace(const himuon_top &) { return 0; }

hipError_t launch_sample(const himuon_sampling &c, void *, hipStream_t stream) {
  SampleParams p{};
  p.uniform = c.uniform;
  p.temperature = c.row_temperature;
  p.top_k = c.row_top_k;
  p.top_p = c.row_top_p;
  p.min_p = c.row_min_p;
  p.token = c.token;
  p.logp = c.logp;
  p.kept = c.kept;
  p.ld_logits = c.ld_logits;
  p.vocab = (int32_t)c.vocab;
  p.k = c.top_k;
  // the sum over a row stays below 2^63
  p.mass_bits = 62 - (64 - __builtin_clzll((u64)c.vocab));
  p.T = c.temperature;
  p.p = c.top_p;
  p.m = c.min_p;
  return c.dtype == HIMUON_BF16 ? launch_sample_t<__bf16>(c, p, stream) : launch_sample_t<float>(c, p, stream);
}

hipError_t launch_top(const himuon_top &c, void *, hipStream_t stream) {
  TopParams p{};
  p.value = c.value;
  p.index = c.index;
  p.rest = c.rest;
  p.ld_logits = c.ld_logits;
  p.ld_top = c.ld_top;
  p.vocab = (int32_t)c.vocab;
  p.k = c.k;
  p.k2 = (float)(kLog2e / c.temperature);
  p.inv_temp = (float)(1. / c.temperature);
  return c.dtype == HIMUON_BF16 ? launch_top_t<__bf16>(c, p, stream) : launch_top_t<float>(c, p, stream);
}

}  // namespace himuon
