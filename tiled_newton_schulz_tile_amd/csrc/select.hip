// Choosing tokens from rows of logits: sampling with temperature, top-k, top-p and min-p from given
// random numbers (himuon_sample), and a row's k largest logits with the log-sum-exp of the others
// (himuon_top_logits).
//
// The order of a row's tokens is from the largest logit to the smallest, and among equal ones by
// index: a token's rank key is a 64-bit number, its logit's bits mapped to grow downwards above its
// index, unlike any other of the row.  Every filter keeps a first part of that order, so it is held
// as the last rank key that it keeps (its border).
//
// A row is read once.  Each of a block's waves goes through a stretch of it on its own: it sums the
// powers, and it appends to a list in LDS what the filters may keep, which most often is a small part
// of the row.  What they may keep is all from a bound on, which rises on the way: the k-th largest
// logit so far, or one below which all tokens together have too little probability to matter.  Borders
// and draw then come from the lists.  Waves meet once, at the end of the row; with many rows a block is
// one wave.  Rows whose lists overflow (flat ones) are read again several times: by blocks of 4 waves or more
// at once, for smaller ones by a second launch.
//
// A border is found by a descent over the digits of the rank key: a histogram of the elements in the
// present range, the bin in which the count (or the probability) reaches its target, and that bin as
// the next range, until one element is left.
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
// before +inf), and back.
__device__ __forceinline__ unsigned down_key(float z) {
  const unsigned u = __builtin_bit_cast(unsigned, z != z ? __builtin_nanf("") : z + 0.f);
  return u ^ ((unsigned)((int)~u >> 31) >> 1);
}
__device__ __forceinline__ float logit_of_key(unsigned down) {
  return __builtin_bit_cast(float, down & 0x80000000u ? down : down ^ 0x7fffffffu);
}
// Rank keys: a logit's number (16 bits of it for bf16) above its index.
constexpr int kIndexBits = 20;
static_assert(HIMUON_TOP_VOCAB <= 1 << kIndexBits, "an index fits");
template <class T>
constexpr int kKeyShift = sizeof(T) == 2 ? 16 : 0;
template <class T>
__device__ __forceinline__ u64 rank_key(float z, int index) {
  return (u64)(down_key(z) >> kKeyShift<T>) << kIndexBits | (unsigned)index;
}
template <class T>
__device__ __forceinline__ float logit_of(u64 r) {
  unsigned down = (unsigned)(r >> kIndexBits) << kKeyShift<T>;
  if (kKeyShift<T> && !(down & 0x80000000u)) down |= 0xffffu;
  return logit_of_key(down);
}
__device__ __forceinline__ int index_of(u64 r) { return (int)(r & (((u64)1 << kIndexBits) - 1)); }
// The first and the last key that a logit can have.
template <class T>
__device__ __forceinline__ u64 first_key(float z) { return rank_key<T>(z, 0); }
template <class T>
__device__ __forceinline__ u64 last_key(float z) { return rank_key<T>(z, 0) | (((u64)1 << kIndexBits) - 1); }

__device__ __forceinline__ float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }   // NaN wins

// Vector `vec` of a row of V elements; -inf stands in for what lies beyond the row.
template <class T>
__device__ __forceinline__ u32x4 row_vector(const T *z, int vec, int V) {
  constexpr int N = Vec<T>::N;
  if ((vec + 1) * N <= V) return Vec<T>::load(z + (int64_t)vec * N);
  u32x4 v = {Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest};
#pragma unroll 1
  for (int at = V - 1; at >= vec * N; --at) {   // (from the back, each moving the others up)
    const unsigned x = __builtin_bit_cast(unsigned, Vec<T>::load1(z + at));
#pragma unroll
    for (int i = 3; i > 0; --i) v[i] = N == 8 ? v[i] << 16 | v[i - 1] >> 16 : v[i - 1];
    v[0] = N == 8 ? v[0] << 16 | x >> 16 : x;
  }
  return v;
}

// LDS accesses of one wave's lanes before this are seen by all of its lanes behind it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
__device__ __forceinline__ u64 wave_scan(u64 x) {   // inclusive
  return __builtin_bit_cast(u64, dev::wave_scan(__builtin_bit_cast(double, x), 0.0, [](double a, double b) {
    return __builtin_bit_cast(double, __builtin_bit_cast(u64, a) + __builtin_bit_cast(u64, b));
  }));
}
__device__ __forceinline__ double wave_scan(double x) {
  return dev::wave_scan(x, 0.0, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ int lanes_before(u64 ballot) {
  return __builtin_amdgcn_mbcnt_hi((unsigned)(ballot >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)ballot, 0));
}
__device__ __forceinline__ int lane_of(u64 ballot) { return __builtin_ctzll(ballot); }
template <class X>
__device__ __forceinline__ X from_lane(X x, int lane) {   // lane: the same in all lanes
  if constexpr (sizeof(X) == 4)
    return __builtin_bit_cast(X, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
  else {
    const u64 u = __builtin_bit_cast(u64, x);
    return __builtin_bit_cast(X, (u64)(unsigned)__builtin_amdgcn_readlane((int)(u >> 32), lane) << 32 |
                                     (unsigned)__builtin_amdgcn_readlane((int)u, lane));
  }
}

// A histogram of a descent.
template <int BINS>
struct Histogram {
  u64 mass[BINS];
  unsigned count[BINS];
};
// What is left of a descent's range of rank keys, and what weighs before it.
struct Range {
  u64 first, last, before;
};
// bin_shift: the keys of a bin of `bits` digits.
__device__ __forceinline__ int bin_shift(const Range &r, int digits) {
  const int bits = 64 - __builtin_clzll((r.last - r.first) | 1);
  return bits > digits ? bits - digits : 0;
}
// The bin where the target is reached becomes the range; whether that is the end: one key, or one element.
__device__ __forceinline__ bool narrow(Range &r, int bin, u64 before, unsigned count, int shift) {
  r.first += (u64)bin << shift;
  const u64 width = ((u64)1 << shift) - 1;
  r.last = r.last - r.first < width ? r.last : r.first + width;
  r.before = before;
  return shift == 0 || count == 1;
}

// The last of n rank keys in LDS (one wave; all between first and last) up to which they weigh the target at
// least: the first one that reaches it; `last` where all weigh less.  weight(key): all together below 2^64.
// target_of(total): the target, 1 or more, given what all weigh.  COUNT: each weighs 1.
constexpr int kWaveBins = 256;
template <bool COUNT, class WEIGHT, class TARGET>
__device__ __forceinline__ u64 find_border(const u64 *list, int n, u64 first, u64 last, WEIGHT weight, TARGET target_of,
                                           Histogram<kWaveBins> &h) {
  constexpr int B = kWaveBins / 64;   // bins a lane
  const int lane = threadIdx.x & 63;
  Range r = {first, last, 0};
  u64 target = 0;
  for (bool top = true;; top = false) {
    const int shift = bin_shift(r, 8);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (!COUNT) h.mass[lane * B + i] = 0;
      h.count[lane * B + i] = 0;
    }
    wave_sync();
    for (int j = lane; j < n; j += 64) {
      const u64 key = list[j];
      if (key < r.first || key > r.last) continue;
      const int bin = (int)((key - r.first) >> shift);
      atomicAdd(&h.count[bin], 1u);
      if (!COUNT) atomicAdd(&h.mass[bin], weight(key));
    }
    wave_sync();
    u64 w[B], mine = 0;
#pragma unroll
    for (int i = 0; i < B; ++i) mine += w[i] = COUNT ? h.count[lane * B + i] : h.mass[lane * B + i];
    const u64 upto = wave_scan(mine);
    if (top) target = target_of(from_lane(upto, 63));
    const u64 hit = __ballot(r.before + upto >= target);
    if (hit == 0) return last;
    u64 at = r.before + upto - mine;
    int bin = 0;
#pragma unroll
    for (int i = 0; i < B - 1; ++i)
      if (bin == i && at + w[i] < target) {
        at += w[i];
        bin = i + 1;
      }
    const int l = lane_of(hit);
    bin = l * B + from_lane(bin, l);
    if (narrow(r, bin, from_lane(at, l), h.count[bin], shift)) return r.last;
    wave_sync();
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
// Powers 2^((z - ref) k) for logits that are not far above ref (2^100 times its power); 2^-1010 at least: those
// below kNoPower are none.
//
// The distance to ref is taken in fp64, first of all: powers and sums relative to references of any size are what
// these are apart.  The product and its fraction come from fused multiply-adds, so the error of a power is that of k
// and of the polynomial.  ref's own power is 1 exactly, and sums over logits that equal it are whole numbers: a border
// that falls between two of them does so here.
constexpr double kNoPower = 0x1p-1000;
struct Powers {
  double k, ref, low;   // low: the least distance
  double unit;          // multiples of 1 / unit in histograms
  __device__ __forceinline__ void refer_to(float to, double to_k) {
    k = to_k;
    ref = to;
    low = -1009. * (1.00001 * __builtin_amdgcn_rcp(k));   // (its power is between 2^-1010.1 and 2^-1008.9)
  }
  __device__ __forceinline__ double of(float z) const {
    constexpr double kWhole = 0x1.8p52;   // (a sum with it ends in a whole number, the power's exponent)
    const double d = __builtin_fmax((double)z - ref, low);
    const double a = __builtin_fma(d, k, kWhole), f = __builtin_fma(d, k, kWhole - a);
    const u64 p = __builtin_bit_cast(u64, pow2_fraction(f));
    const unsigned hi = (unsigned)(p >> 32) + ((unsigned)__builtin_bit_cast(u64, a) << 20);
    return __builtin_bit_cast(double, (u64)hi << 32 | (unsigned)p);
  }
  __device__ __forceinline__ u64 mass(float z) const { return (u64)(of(z) * unit + 0.5); }
  // What powers relative to `from`, a logit that is not above ref, have to be multiplied with to be relative to ref.
  __device__ __forceinline__ double scale_from(float from) const {
    const double x = of(from);
    return x < kNoPower ? 0. : x;
  }
};

// top: the row's largest logit; all, kept: sums of powers relative to it.
__device__ __forceinline__ void write_token(const SampleParams &p, int64_t row, const Settings &s, int token, float logit,
                                            float top, double all, double kept) {
  gmem(p.token)[row] = token;
  gmem(p.logp)[row] = s.greedy ? 0.f : (float)(((double)logit - top) * (s.k * 0.69314718055994530942) - log(all));
  gmem(p.kept)[row] = s.greedy ? 1.f : (float)(kept / all);
}

// What a row's filters keep, once their borders are known.
template <class T>
struct Kept {
  u64 border;       // the last rank key of top_k and top_p
  double least;     // the least power of min_p, kNoPower at least
  __device__ __forceinline__ double power(const Powers &e, int index, float z) const {
    const double x = e.of(z);
    return rank_key<T>(z, index) <= border && x >= least ? x : 0.;
  }
};

// The target of top_p in multiples of 1 / unit: what its first tokens have to reach.  total: of those that top_k
// keeps, or else all, the sum of the row's powers.
__device__ __forceinline__ u64 target_of_p(const Settings &s, const Powers &e, u64 total, double all) {
  const double t = __builtin_ceil(s.top_p * (s.by_k ? (double)total : all * e.unit));
  return t < 1. ? (u64)1 : (u64)t;
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
__device__ __forceinline__ float wave_maximum(float x) {
  return wave_reduce(x, -__builtin_inff(), [](float a, float b) { return maximum(a, b); });
}

// One wave: which of n parts (0 or more each, in order) the target falls into: the first one up to
// which they sum to more; the last that is not 0 if none does.  before: the sum before it.
template <class PART>
__device__ __forceinline__ int find_part(int n, double target, PART part, double &before) {
  const int lane = threadIdx.x & 63;
  double sum = 0;
  int last = 0;
  before = 0;
  for (int c = 0; c < n; c += 64) {
    const double w = c + lane < n ? part(c + lane) : 0., s = wave_scan(w);
    const u64 hit = __ballot(w > 0. && sum + s > target), some = __ballot(w > 0.);
    if (hit || some) {
      const int l = hit ? lane_of(hit) : 63 - __builtin_clzll(some);
      last = c + l;
      before = sum + from_lane(s - w, l);
      if (hit) break;
    }
    sum += from_lane(s, 63);
  }
  return last;
}

// ---- one wave's stretch of a row
constexpr int kTurnVecs = 4;                  // vectors a lane has at a time
constexpr int kTurn = 64 * kTurnVecs;         // vectors a wave has at a time
constexpr int kTurns = 64;                    // turns of a stretch at most
constexpr int kListMost = 768;                // keys of a list
constexpr int kFirstTurns = 4;
constexpr int kQuota = 224;                   // rank of the logit that the bound follows, at most
constexpr float kFar = 100.f;                 // octaves

// What a wave's stretch comes to.
struct Stretch {
  float top;       // its largest logit (NaN: there is one)
  float ref;       // the logit that its sums are relative to (-inf: no logit)
  double sum;      // of the powers of what is not in the list
  double listed;   // and of what is
  float raised;    // what quota raised the bound to (-FLT_MAX: it did not)
  float last_bound;   // sweep()
  int n;           // keys in the list; kListMost + 1: they did not fit
};

// What the list of a stretch has to hold, and how its sum is taken.
struct Wants {
  int quota;             // 0, or: the quota largest
  int most, then;        // keys of the list above which the bound is raised: in the first kFirstTurns, and then
  double k, temp;        // log2(e) / temperature, temperature
  double share_p;        // 0, or: all tokens but some with less than this share of all probability
  double share_m;        // 0, or: all tokens with at least this share of the largest's probability
  bool none;             // nothing
};
// The bound that comes from the largest logit top, and from what all powers relative to ref sum to at least.  Below
// what the formulas give: the share and its logarithm are fp32, which is 2^-22 of a temperature together where the share
// is near 1 and its logarithm near 0, and 2^-22 of the step elsewhere; sums and products are off by 2^-23 of their terms.
__device__ __forceinline__ float bound_of(const Wants &want, float top, float ref, double sum, int V) {
  const auto below = [&](float from, double share) {
    const float temp = (float)want.temp, step = temp * kLn2 * __builtin_amdgcn_logf((float)share);   // (negative)
    const float room = 1e-5f * (__builtin_fabsf(from) + __builtin_fabsf(step)) + 0x1p-20f * temp;
    return __builtin_fmaxf(from + step - room, -__FLT_MAX__);
  };
  float b = -__FLT_MAX__;
  if (want.share_p > 0.) b = __builtin_fmaxf(b, below(ref, __builtin_fmin(want.share_p * sum / V, 1e30)));
  if (want.share_m > 0.) b = __builtin_fmaxf(b, below(top, want.share_m));
  return __builtin_fminf(b, top);
}

// A number that `quota` at least of N values a lane are not below, and where ties allow it no more than
// quota + quota / 8 + 8; -inf where there are not so many above that.  By halves of the values' range, and
// where that does not converge (a mask among them) of their keys' range.
template <int N>
__device__ __forceinline__ float nth_largest(const float (&x)[N], int quota) {
  float most = x[0], least = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) {
    most = __builtin_fmaxf(most, x[i]);
    least = __builtin_fminf(least, x[i]);
  }
  const auto count = [&](float t) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) c += __builtin_popcountll(__ballot(x[i] >= t));
    return c;
  };
  float hi = wave_max(most), lo = __builtin_fmaxf(-wave_max(-least), -__FLT_MAX__);   // (fewer from hi on, enough from lo on)
  if (count(hi) >= quota) return hi;
  if (count(lo) < quota) return -__builtin_inff();
  for (int turn = 0;; ++turn) {
    float mid = lo * 0.5f + hi * 0.5f;
    if (turn >= 16) {
      const unsigned a = down_key(hi), b = down_key(lo);
      mid = logit_of_key(a + (b - a) / 2);
    }
    if (!(mid > lo && mid < hi)) {
      if (turn >= 16) return lo;
      continue;
    }
    const int c = count(mid);
    if (c >= quota) {
      lo = mid;
      if (c <= quota + quota / 8 + 8) return lo;
    } else {
      hi = mid;
    }
  }
}
// The same of a list, of a short one in fewer steps (4096 x 128256 bf16, k = 64: 295 us, 310 us without).
template <class T, int N>
__device__ __forceinline__ float nth_of_keys(const u64 *list, int n, int quota) {
  float x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = i * 64 + (threadIdx.x & 63);
    x[i] = j < n ? logit_of<T>(list[j]) : -__builtin_inff();
  }
  return nth_largest(x, quota);
}
template <class T>
__device__ __forceinline__ float nth_of_list(const u64 *list, int n, int quota) {
  if (n <= 320) return nth_of_keys<T, 5>(list, n, quota);
  return nth_of_keys<T, kListMost / 64>(list, n, quota);
}

// x[e], e a lane's own.
template <int N>
__device__ __forceinline__ float pick_element(const float (&x)[N], int e) {
  float a[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float low = x[2 * i], high = x[2 * i + 1];   // (values: a choice of places would put x in memory)
    a[i] = e & 1 ? +high : +low;
  }
  if constexpr (N == 2) return a[0];
  else return pick_element(a, e >> 1);
}
// Appends a vector's elements from `least` on (finite: the vectors behind a row are -inf) to the wave's list of n keys
// (of which kListMost are kept; n counts on), in the order of their indices.  A lane mostly has one at most: one turn
// of the loop (4096 x 128256 bf16, k = 64: 310 us then, and 335 us with a step for each of a vector's elements).
template <class T, int N>
__device__ __forceinline__ void append(u64 *list, int &n, int at, const float (&x)[N], float least) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) m |= x[e] >= least ? 1u << e : 0u;
  const u64 any = __ballot(m != 0);
  int pos = n + lanes_before(any);
  n += __builtin_popcountll(any);
  if (__any(m & (m - 1))) {   // lanes with several
    const int more = __builtin_popcount(m) - 1;
#pragma unroll
    for (int b = 0; 1 << b < N; ++b) {
      const u64 with = __ballot(more > 0 && (more >> b & 1));
      pos += lanes_before(with) << b;
      n += __builtin_popcountll(with) << b;
    }
  }
  while (m) {
    const int e = __builtin_ctz(m);
    if (pos < kListMost) list[pos] = rank_key<T>(pick_element(x, e), at + e);
    ++pos;
    m &= m - 1;
  }
}

template <class T>
struct Turn {
  u32x4 v[kTurnVecs];
  __device__ __forceinline__ void load(const T *z, int turn, int V) {
    const int at = turn * kTurn + (threadIdx.x & 63);
    if ((turn + 1) * kTurn * Vec<T>::N <= V) {
#pragma unroll
      for (int i = 0; i < kTurnVecs; ++i) v[i] = Vec<T>::load(z + (int64_t)(at + 64 * i) * Vec<T>::N);
    } else {
#pragma unroll
      for (int i = 0; i < kTurnVecs; ++i) v[i] = row_vector(z, at + 64 * i, V);
    }
  }
  // Vector i, the same in all lanes (a choice of registers, so that loops over vectors stay loops).
  __device__ __forceinline__ u32x4 pick(int i) const {
    static_assert(kTurnVecs == 4, "four vectors");
    const bool odd = i & 1, high = i & 2;
    u32x4 a;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned x = odd ? v[1][j] : v[0][j], y = odd ? v[3][j] : v[2][j];
      a[j] = high ? y : x;
    }
    hold_packed(a);
    return a;
  }
};

// The largest logit of each of a lane's vectors, and of all of them.
template <class T>
__device__ __forceinline__ float turn_maximum(Turn<T> &turn, float (&most)[kTurnVecs]) {
  constexpr int N = Vec<T>::N;
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kTurnVecs; ++i) {
    hold_packed(turn.v[i]);
    float x[N];
    Vec<T>::unpack(turn.v[i], x);
    most[i] = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) most[i] = maximum(most[i], x[j]);
    top = maximum(top, most[i]);
    hold_packed(turn.v[i]);
  }
  return top;
}
// f(a lane's vector, its elements) for all vectors of a row in memory, 64 consecutive ones a wave and call.
template <class T, int THR, class F>
__device__ __forceinline__ void each_vector(const T *z, int V, F f) {
  const int lane = threadIdx.x & 63, turns = ((V + Vec<T>::N - 1) / Vec<T>::N + kTurn - 1) / kTurn;
  for (int t = threadIdx.x >> 6; t < turns; t += THR / 64) {
    Turn<T> now;
    now.load(z, t, V);
#pragma unroll 1
    for (int i = 0; i < kTurnVecs; ++i) {
      float x[Vec<T>::N];
      Vec<T>::unpack(now.pick(i), x);
      f(t * kTurn + i * 64 + lane, x);
    }
  }
}

// find_border() among the elements of a row of V in memory, by the THR threads of a block.  A bin that is a
// single logit's (in bf16 mostly all are) has its elements counted, and its mass comes from their number.
template <int THR>
struct BlockLds {
  Histogram<4 * THR> h;
  u64 wave[THR / 64];
  int bin;
  u64 before;
  unsigned count;
};
template <class T, int THR, bool COUNT, class WEIGHT, class TARGET>
__device__ __forceinline__ u64 find_border_in_row(const T *z, int V, u64 first, u64 last, WEIGHT weight, TARGET target_of,
                                                  BlockLds<THR> &lds) {
  constexpr int N = Vec<T>::N, B = 4, kDigits = 31 - __builtin_clz(B * THR);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  Range r = {first, last, 0};
  u64 target = 0;
  for (bool top = true;; top = false) {
    const int shift = bin_shift(r, kDigits);
    const bool single = COUNT || (sizeof(T) == 2 && shift <= 20);
    for (int i = tid; i < B * THR; i += THR) {
      lds.h.mass[i] = 0;
      lds.h.count[i] = 0;
    }
    if (tid == 0) lds.bin = -1;
    __syncthreads();
    const float most = logit_of<T>(r.first), least = logit_of<T>(r.last);   // (a NaN is above everything)
    each_vector<T, THR>(z, V, [&](int at, float (&x)[N]) {
      bool in = false;
#pragma unroll
      for (int e = 0; e < N; ++e) in = in || !(x[e] < least || x[e] > most);
      if (!__any(in)) return;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const u64 key = rank_key<T>(x[e], at * N + e);
        if (key < r.first || key > r.last || at * N + e >= V) continue;
        const int bin = (int)((key - r.first) >> shift);
        atomicAdd(&lds.h.count[bin], 1u);
        if (!single) atomicAdd(&lds.h.mass[bin], weight(x[e]));
      }
    });
    __syncthreads();
    u64 have[B], mine = 0;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int bin = tid * B + i;
      const unsigned n = lds.h.count[bin];
      have[i] = COUNT ? n : !single ? lds.h.mass[bin] : n > 0 ? n * weight(logit_of<T>(r.first + ((u64)bin << shift))) : 0;
      mine += have[i];
    }
    u64 upto = wave_scan(mine);
    if (lane == 63) lds.wave[w] = upto;
    __syncthreads();
    u64 total = 0;
    for (int i = 0; i < THR / 64; ++i) {
      if (i < w) upto += lds.wave[i];
      total += lds.wave[i];
    }
    if (top) target = target_of(total);
    u64 at = r.before + upto - mine;
    if (at < target && at + mine >= target) {
      int bin = 0;
#pragma unroll
      for (int i = 0; i < B - 1; ++i)
        if (bin == i && at + have[i] < target) {
          at += have[i];
          bin = i + 1;
        }
      lds.bin = tid * B + bin;
      lds.before = at;
      lds.count = lds.h.count[tid * B + bin];
    }
    __syncthreads();
    const int bin = lds.bin;
    const u64 before = lds.before;
    const unsigned count = lds.count;
    __syncthreads();
    if (bin < 0) return last;
    if (narrow(r, bin, before, count, shift)) return r.last;
  }
}

// A wave goes through turns [t0, t1) of a row, the first of which is in `now`, with a first logit that
// powers are relative to and a first bound (which hold for the row).  exact: powers in fp64; else in fp32.
// They are relative to a logit that follows the largest by kFar, and if CEIL (fp32 alone) to the bound, above which
// nothing is summed.  turns: nullptr, or what each turn weighs.  last_quota: rank of the
// logit in the final list that last_bound is not above (0: none).
template <class T, bool CEIL>
__device__ __forceinline__ Stretch sweep(Turn<T> &now, const T *z, int V, int t0, int t1, const Wants &want, bool exact,
                                         float ref, float bound, u64 *list, double *turns, int last_quota) {
  constexpr int N = Vec<T>::N;
  const int lane = threadIdx.x & 63;
  const float k32 = (float)want.k, far = (float)(kFar / want.k);
  // (the second part of k, above 0: the product of -inf with it is -inf, too)
  const float hi = CEIL ? k32 : __builtin_bit_cast(float, __builtin_bit_cast(unsigned, k32) - 1), lo = (float)(want.k - hi);
  Stretch out = {-__builtin_inff(), -__builtin_inff(), 0., 0., -__FLT_MAX__, -__FLT_MAX__, 0};
  if (want.none) bound = __builtin_inff();
  float largest = -__builtin_inff();
  bool stop = false;
  double sum = 0, part = 0;
  Powers e;
  e.unit = 1.;
  e.refer_to(ref > -__builtin_inff() ? ref : 0.f, want.k);
  const auto refer_to = [&](float to) {
    const bool none = ref == -__builtin_inff();
    e.refer_to(to, want.k);
    const double scale = none ? 0. : e.scale_from(ref);
    sum *= scale;
    part = none ? 0. : part * scale;
    if (turns) turns[lane] *= scale;
    ref = to;
  };
  const auto logit_at = [&](int j) { return logit_of<T>(list[j]); };
  // An element is looked at more closely from here on: it belongs to the list, or the powers' reference has to
  // move (so that none is past 2^100).
  const auto threshold = [&] { return CEIL ? bound : __builtin_fminf(bound, ref + far); };
  float close = threshold();
  const auto vector = [&](int at, float (&x)[N]) {   // at: the index of its first element
    float most = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) most = maximum(most, x[j]);
    largest = maximum(largest, most);
    if (__any(!(most < close))) {
      if (__any(!(most < (CEIL ? __builtin_inff() : ref + far)))) {
        const float top = wave_maximum(most);
        stop = stop || !(top < __builtin_inff());   // NaN or +inf: nothing of the row is needed
        if (!CEIL && !stop && top > -__builtin_inff()) {
          refer_to(top);
          bound = __builtin_fmaxf(bound, bound_of(want, top, top, 1., V));
          close = threshold();
        }
      }
      if (__any(most >= bound)) {
        append<T>(list, out.n, at, x, bound);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = x[j] >= bound ? -__builtin_inff() : x[j];
      }
    }
    if (!CEIL && exact) {
      double s[2];
#pragma unroll
      for (int j = 0; j < N; ++j) s[j & 1] = j < 2 ? e.of(x[j]) : s[j & 1] + e.of(x[j]);
      part += s[0] + s[1];
    } else {
      // (the difference before the product, which then has an error of its own size; in the sampler k has two parts)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float d = x[j] - ref;
        x[j] = __builtin_amdgcn_exp2f(CEIL ? d * hi : __builtin_fmaf(d, hi, d * lo));
      }
#pragma unroll
      for (int d = 1; d < N; d *= 2)
#pragma unroll
        for (int j = 0; j < N; j += 2 * d) x[j] += x[j + d];
      part += (double)x[0];
    }
  };
  if (turns) turns[lane] = 0.;
  for (int t = t0; t < t1; ++t) {
    part = 0;
    const bool more = t + 1 < t1;
    const int first = (t * kTurn + lane) * N;
    const bool whole = (t + 2) * kTurn * N <= V;   // (the next turn)
#pragma unroll
    for (int i = 0; i < kTurnVecs; ++i) {
      float x[N];
      Vec<T>::unpack(now.v[i], x);
      if (more) {   // its place takes the next turn's
        const int at = (t + 1) * kTurn + 64 * i + lane;
        now.v[i] = whole ? Vec<T>::load(z + (int64_t)at * N) : row_vector(z, at, V);
      }
      vector(first + i * 64 * N, x);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (stop || out.n > kListMost) {
      out.top = wave_maximum(largest);
      if (stop) out.n = 0;
      return out;
    }
    if (ref == -__builtin_inff()) part = 0;   // (no logits so far)
    if (turns) {
      part = part < 0x1p-980 ? 0. : part;   // (nothing but powers that are none)
      const double all = wave_sum(part);
      if (lane == 0) turns[t - t0] = all;
    }
    sum += part;
    part = 0;
    const int most = t - t0 < kFirstTurns ? want.most : want.then;
    while (out.n > most || (!more && last_quota > 0 && out.n >= last_quota)) {
      const bool raise = out.n > most;
      wave_sync();
      float b;
      if (want.quota > 0) {
        b = nth_of_list<T>(list, out.n, raise ? want.quota : last_quota);
      } else {
        double all = sum;
        for (int j = lane; j < out.n; j += 64) all += e.of(logit_at(j));
        b = bound_of(want, wave_maximum(largest), ref, wave_sum(all), V);
      }
      b = __builtin_fmaxf(bound, b);
      if (!raise) {
        out.last_bound = b;
        break;
      }
      // the bound rises, and what is below it is dropped
      bound = b;
      if (want.quota > 0) out.raised = b;
      if (CEIL && b > ref) refer_to(b);   // (an fp32 power loses 2^-22 by each octave that it is away)
      close = threshold();
      int n = 0;
      for (int j = 0; j < out.n; j += 64) {
        const u64 r = j + lane < out.n ? list[j + lane] : 0;
        const float x = logit_of<T>(r);
        const bool in = j + lane < out.n, stays = in && x >= bound;
        const u64 stay = __ballot(stays);
        if (stays) list[n + lanes_before(stay)] = r;
        if (in && !stays) sum += e.of(x);
        n += __builtin_popcountll(stay);
      }
      out.n = n;
      wave_sync();
      if (n > most) {   // (more of them than a list is for)
        out.n = kListMost + 1;
        return out;
      }
    }
  }
  out.top = wave_maximum(largest);
  out.ref = ref;
  out.sum = wave_sum(sum);
  if (!CEIL && out.n > 0) {
    wave_sync();
    double all = 0;
    for (int j = lane; j < out.n; j += 64) all += e.of(logit_at(j));
    out.listed = wave_sum(all);
  }
  return out;
}

// Keys of a list at which the bound is raised to its quota-th largest (which leaves quota + quota / 8 + 8
// of them): often while it rises, and with room for those of another turn, some quota in the beginning and a
// quarter of the list at most after kFirstTurns (with the first room all along the top 449 of 4096 x 128256 bf16 take
// 847 us, and not 686: the bound is raised every 28 keys).
__device__ __forceinline__ int raise_at(int quota, bool first) {
  const int often = 2 * quota + 64, room = first ? kListMost - 2 * quota - 32 : kListMost * 3 / 4;
  return often < room ? often : room;
}
// A row's stretches: W waves, turns [0, turns) of the row in W parts.
__device__ __forceinline__ int stretch_turn(int turns, int w, int W) { return (int)((int64_t)turns * w / W); }
template <class T>
__device__ __forceinline__ int turns_of(int V) {
  return ((V + Vec<T>::N - 1) / Vec<T>::N + kTurn - 1) / kTurn;
}

// A row's largest logit, by the THR threads of a block, and the sum of all powers, relative to it.  top: NaN or +inf
// or all of them -inf: no sum.
template <class T, int THR>
__device__ __forceinline__ double measure_row(const T *z, const Settings &s, const SampleParams &p, float &top, Powers &e,
                                              double *wave) {
  constexpr int N = Vec<T>::N, W = THR / 64;
  const int lane = threadIdx.x & 63;
  top = -__builtin_inff();
  each_vector<T, THR>(z, p.vocab, [&](int, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) top = maximum(top, x[i]);
  });
  top = wave_maximum(top);
  __syncthreads();
  if (lane == 0) wave[threadIdx.x >> 6] = top;
  __syncthreads();
  top = wave_maximum((float)wave[lane % W]);
  if (!(__builtin_fabsf(top) < __builtin_inff())) return 0.;
  e.refer_to(top, s.k);
  double all = 0;
  each_vector<T, THR>(z, p.vocab, [&](int, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) all += e.of(x[i]);
  });
  return block_sum_in_order<THR>(all, wave);
}

// The token of a row that is read from memory for every pass over it, by the THR threads of a block.  e: relative to
// its largest logit top; all: the sum of its powers; bound: what is below it is not kept.  chunk: LDS, one for each
// 64 vectors of the row (it may be in the histogram's place).
template <class T, int THR>
__device__ __forceinline__ void sample_from_memory(const T *z, const Settings &s, int64_t row, const SampleParams &p,
                                                   const Powers &e, float top, double all, float bound, BlockLds<THR> &lds,
                                                   double *chunk) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x, lane = tid & 63, V = p.vocab, vecs = (V + N - 1) / N;
  u64 border = last_key<T>(bound);
  if (s.by_k)
    border = find_border_in_row<T, THR, true>(z, V, first_key<T>(top), border, [](float) { return (u64)1; },
                                              [&](u64) { return (u64)s.top_k; }, lds);
  if (s.by_p)
    border = find_border_in_row<T, THR, false>(z, V, first_key<T>(top), border, [&](float x) { return e.mass(x); },
                                               [&](u64 total) { return target_of_p(s, e, total, all); }, lds);
  const Kept<T> kept = {border, __builtin_fmax(s.min_p, kNoPower)};
  const float edge = logit_of<T>(border);   // (of the last token that is kept)
  const auto weigh = [&](int vec, const float (&x)[N]) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < N; ++i) any = any || x[i] >= edge;
    double t = 0;
    if (__any(any)) {
#pragma unroll
      for (int i = 0; i < N; ++i) t += kept.power(e, vec * N + i, x[i]);
    }
    return t;
  };
  // the draw: a wave's 64 vectors are consecutive, so the chunks are in order
  const int chunks = (vecs + 63) / 64;
  each_vector<T, THR>(z, V, [&](int at, float (&x)[N]) {
    const double sum = wave_sum(weigh(at, x));
    if (lane == 0 && at < vecs) chunk[at / 64] = sum;
  });
  __syncthreads();
  if (tid >= 64) return;   // (they wait for the first wave at the next row)
  double total = 0;
  for (int c = lane; c < chunks; c += 64) total += chunk[c];
  total = wave_sum(total);
  const double target = uniform_of(p, row) * total;
  double before, more, last;
  const int c = find_part(chunks, target, [&](int i) { return chunk[i]; }, before);
  float x[N];
  Vec<T>::unpack(row_vector(z, c * 64 + lane, V), x);
  const double own = weigh(c * 64 + lane, x);
  const int v = c * 64 + find_part(64, target - before, [&](int) { return own; }, more);
  const int n = N < V - v * N ? N : V - v * N;
  const float mine = Vec<T>::load1(z + (lane < n ? v * N + lane : V - 1));
  const int i = find_part(n, target - before - more, [&](int j) { return kept.power(e, v * N + j, mine); }, last);
  if (lane == i) write_token(p, row, s, v * N + i, mine, top, all, total);
}

// Whether a block of W waves reads its row again itself where the row's lists do not hold what is asked for.  The
// alternative is a second launch, in blocks of 16 waves, that finds the rows that the first one marked; every call pays
// for it, with such a row or without.
//   Blocks of 4 waves on read again: 1 x 32000 bf16, top_k 23.0 us, and 29.9 with a second launch; 2000 x 32000, top_p 82
//   and 99.
//   Blocks of 1 and 2 waves leave it to the second launch, since one wave takes long over a row: 4096 x 32000, top_k with
//   one flat row 227 us, and 321 where its wave reads again (without a flat row 133 and 115).
constexpr bool again(int W) { return W >= 4; }

template <int W>
struct RowLds {
  static constexpr int kJoined = W == 1 ? 512 : W < 8 ? 1024 : 2048;   // keys of the joined list
  static constexpr int kRanked = W == 1 ? 192 : 512;    // and those that are ranked by counting
  union {
    u64 list[W][kListMost];
    double turns[W][kTurns];
    std::conditional_t<again(W), BlockLds<64 * W>, u64> block;
    double chunk[W][kListMost];
  };
  u64 joined_list[W == 1 ? 1 : kJoined];
  union {
    Histogram<kWaveBins> wave;
    u64 sorted[kRanked];
  };
  Stretch out[W];
  Settings settings;
  double part[W];
  float first_top[W], first_bound[W], raised[W], last_bound[W];
  int count[W];
  __device__ __forceinline__ u64 *joined() { return W == 1 ? &list[0][0] : joined_list; }
};

// The n-th largest of W numbers in LDS, one wave.
template <int W>
__device__ __forceinline__ float nth_bound(const float *bound, int n) {
  if constexpr (W == 1) return bound[0];
  const int lane = threadIdx.x & 63;
  const float mine = lane < W ? bound[lane] : -__builtin_inff();
  int rank = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float b = from_lane(mine, i);
    rank += b > mine || (b == mine && i < lane) ? 1 : 0;
  }
  return from_lane(mine, lane_of(__ballot(lane < W && rank == n - 1)));
}

// How W waves find a bound that is not above the k-th largest logit of all: each takes its quota-th
// largest (a little more than its share of k), and `ranks` of them have quota logits from their bounds on, k together.
// More ranks than waves: no bound.
struct Shares {
  int quota, ranks;
};
template <int W>
__device__ __forceinline__ Shares shares_of(int k) {
  if (k <= 0) return {0, 1};
  int q = W == 1 ? k : (k + k / 4 + W - 1) / W + 1;
  q = q < kQuota ? q : kQuota;
  // (a quotient below 2^20 by fp32: half a unit off a whole number before it is cut off)
  return {q, (int)(((float)(k + q - 1) + 0.5f) * __builtin_amdgcn_rcpf((float)q))};
}

// What a block knows of a row from its waves' first turns: the largest logit, and a bound for its k
// largest.  Every wave calls it.
template <class T, int W>
__device__ __forceinline__ void first_bounds(Turn<T> &now, Shares share, RowLds<W> &lds, float &top, float &bound) {
  float most[kTurnVecs];
  top = wave_maximum(turn_maximum(now, most));
  bound = -__FLT_MAX__;
  const bool any = share.quota > 0 && share.ranks <= W;
  if (any && top < __builtin_inff()) bound = __builtin_fmaxf(bound, nth_largest(most, share.quota));
  if constexpr (W > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      lds.first_top[w] = top;
      lds.first_bound[w] = bound;
    }
    __syncthreads();
    top = wave_maximum(lds.first_top[(threadIdx.x & 63) < W ? threadIdx.x & 63 : 0]);
    if (any) bound = nth_bound<W>(lds.first_bound, share.ranks);
  }
}
// What a wave leaves of its stretch for the others; the block waits behind it.
template <int W>
__device__ __forceinline__ void leave_stretch(const Stretch &mine, RowLds<W> &lds) {
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    lds.out[w] = mine;
    lds.raised[w] = mine.raised;
    lds.last_bound[w] = mine.last_bound;
  }
  __syncthreads();
}
// What the stretches come to together: every wave calls it, lane i has the i-th stretch's reference, sum and
// sum with what is listed (lanes from W on: none).
struct Together {
  float top;
  bool fits;
  int listed;
  float ref;
  double sum, all;
};
template <int W>
__device__ __forceinline__ Together together(const RowLds<W> &lds) {
  const int lane = threadIdx.x & 63;
  const Stretch &x = lds.out[lane < W ? lane : 0];
  const bool in = lane < W;
  Together t;
  t.top = wave_maximum(in ? x.top : -__builtin_inff());
  t.fits = __ballot(in && x.n > kListMost) == 0;
  t.listed = (int)wave_reduce(in ? (unsigned)x.n : 0u, 0u, [](unsigned a, unsigned b) { return a + b; });
  t.ref = in ? x.ref : -__builtin_inff();
  t.sum = in ? x.sum : 0.;
  t.all = in ? x.sum + x.listed : 0.;
  return t;
}

// The stretches' lists, from bound on, in one, in their order; its length, or kJoined + 1 where it does
// not fit.  Every wave calls it; the block waits at its end.
template <class T, int W>
__device__ __forceinline__ int join_lists(RowLds<W> &lds, float bound) {
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, n = lds.out[w].n;
  const u64 *list = lds.list[w];
  int at = 0, total = 0;
  if constexpr (W > 1) {
    int mine = 0;
    for (int j = 0; j < n; j += 64) {
      const u64 r = j + lane < n ? list[j + lane] : ~(u64)0;
      mine += __builtin_popcountll(__ballot(j + lane < n && logit_of<T>(r) >= bound));
    }
    if (lane == 0) lds.count[w] = mine;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i < w) at += lds.count[i];
      total += lds.count[i];
    }
    if (total > RowLds<W>::kJoined) return RowLds<W>::kJoined + 1;
  }
  for (int j = 0; j < n; j += 64) {   // (one wave's list is shortened in its place)
    const u64 r = j + lane < n ? list[j + lane] : ~(u64)0;
    const bool in = j + lane < n && logit_of<T>(r) >= bound;
    const u64 all = __ballot(in);
    if (in) lds.joined()[at + lanes_before(all)] = r;
    at += __builtin_popcountll(all);
  }
  __syncthreads();
  if constexpr (W == 1) return at <= RowLds<W>::kJoined ? at : RowLds<W>::kJoined + 1;
  return total;
}
// How many of n keys have a logit of `least` or more (one wave).
template <class T>
__device__ __forceinline__ int count_from(const u64 *keys, int n, float least) {
  int c = 0;
  for (int j = threadIdx.x & 63; j - (int)(threadIdx.x & 63) < n; j += 64)
    c += __builtin_popcountll(__ballot(j < n && logit_of<T>(keys[j < n ? j : 0]) >= least));
  return c;
}
// How many of n keys are below r.
__device__ __forceinline__ int rank_among(const u64 *keys, int n, u64 r) {
  int rank = 0, i = 0;
  for (; i + 8 <= n; i += 8) {   // (eight reads in flight)
    u64 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = keys[i + j];
#pragma unroll
    for (int j = 0; j < 8; ++j) rank += x[j] < r ? 1 : 0;
  }
  for (; i < n; ++i) rank += keys[i] < r ? 1 : 0;
  return rank;
}

// W waves take a row.  later: the rows that small blocks cannot do are marked there for the second launch.
template <class T, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(W == 2 ? 3 : 4)))
void sample_kernel(const T *logits, SampleParams p, int32_t *later) {
  constexpr int N = Vec<T>::N;
  __shared__ RowLds<W> lds;
  const int64_t row = blockIdx.x;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, V = p.vocab, turns = turns_of<T>(V);
  const T *z = logits + row * p.ld_logits;
  const int t0 = stretch_turn(turns, w, W), t1 = stretch_turn(turns, w + 1, W);
  Turn<T> now;
  now.load(z, t0 < t1 ? t0 : turns, V);
  Settings s = settings_of(p, row);
  if (!again(W) && threadIdx.x == 0) gmem(later)[row] = 0;
  if (!s.good) {
    if (threadIdx.x == 0) write_bad(p, row);
    return;
  }
  const bool everything = !s.by_k && !s.by_p && s.min_p == 0., exact = everything || (s.by_p && !s.by_k);
  const int quota = s.by_k ? s.top_k < kQuota ? s.top_k : kQuota : 0;
  const Shares share = shares_of<W>(s.by_k ? s.top_k : 0);
  const int full = kListMost - 256;
  const Wants want = {quota, quota > 0 ? raise_at(quota, true) : full, quota > 0 ? raise_at(quota, false) : full, s.k, s.temp,
                      s.by_p && !s.by_k ? 1. - s.top_p : 0., s.by_k && s.by_p ? 0. : s.min_p, everything};
  float top, bound;
  first_bounds<T, W>(now, share, lds, top, bound);
  if (!(top < __builtin_inff())) {
    if (threadIdx.x == 0) write_bad(p, row);
    return;
  }
  if (top > -__builtin_inff()) bound = __builtin_fmaxf(bound, bound_of(want, top, top, 1., V));
  if (threadIdx.x == 0) lds.settings = s;   // (for what follows the sweep, which has no registers to spare)
  const Stretch mine = sweep<T, false>(now, z, V, t0, t1, want, exact, top, bound, lds.list[w],
                                                  everything ? lds.turns[w] : nullptr,
                                                  turns > W && share.ranks <= W ? share.quota : 0);
  leave_stretch<W>(mine, lds);
  s = lds.settings;
  const Together row_of = together(lds);
  top = row_of.top;
  bool fits = row_of.fits;
  if (fits && !(__builtin_fabsf(top) < __builtin_inff())) {   // NaN or +inf in the row, nothing but -inf
    if (threadIdx.x == 0) write_bad(p, row);
    return;
  }
  Powers e;
  e.refer_to(top, s.k);
  e.unit = __builtin_amdgcn_ldexp(1., p.mass_bits);
  const double relative = e.scale_from(row_of.ref);   // (a stretch's powers to the row's; 0 without logits)
  const double part_of_all = row_of.all * relative, all = wave_sum(part_of_all);
  if (everything) {
    if (w > 0) return;
    // what each stretch weighs, then the turns of one, the vectors of one turn, the elements of one vector.  A stretch
    // (64 turns) or turn (2^11 elements) that weighs too little to be sure of a turn or an element with a power is none
    const auto some = [](double w, double least) { return w < least ? 0. : w; };
    const Kept<T> kept = {~(u64)0, kNoPower};
    const double target = uniform_of(p, row) * all;
    double before, more, last;
    const int in = find_part(W, target, [&](int) { return some(part_of_all, 0x1p-970); }, before);
    const double scale = from_lane(relative, in);
    const int s0 = stretch_turn(turns, in, W), s1 = stretch_turn(turns, in + 1, W);
    const int turn =
        s0 + find_part(s1 - s0, target - before, [&](int i) { return some(lds.turns[in][i] * scale, 0x1p-980); }, more);
    now.load(z, turn, V);
    double left = target - before - more, seen_left = 0;
    int v = -1, seen = 0;
#pragma unroll 1
    for (int i = 0; i < kTurnVecs && v < 0; ++i) {
      float x[N];
      Vec<T>::unpack(now.pick(i), x);
      double own = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) own += kept.power(e, 0, x[j]);
      const double total = wave_sum(own);
      if (total > 0.) {
        double past;
        seen = (turn * kTurnVecs + i) * 64 + find_part(64, left, [&](int) { return own; }, past);
        seen_left = left - past;
        if (total > left) v = seen;
      }
      left -= total;
    }
    if (v < 0) v = seen;   // (the target is the whole sum, to within its rounding)
    const int n = N < V - v * N ? N : V - v * N;
    const float x = Vec<T>::load1(z + (lane < n ? v * N + lane : V - 1));
    const int i = find_part(n, seen_left, [&](int) { return kept.power(e, 0, x); }, last);
    if (lane == i) write_token(p, row, s, v * N + i, x, top, all, all);
    return;
  }
  int n = 0;
  bound = bound_of(want, top, top, all, V);
  if (fits) {
    if (quota > 0 && share.ranks <= W) bound = __builtin_fmaxf(bound, nth_bound<W>(lds.last_bound, share.ranks));
    n = join_lists<T>(lds, bound);
    fits = n <= RowLds<W>::kJoined;
    // (where a stretch's list followed its kQuota-th largest, the lists hold what is not below what that raised its bound
    // to: enough where that is not above the bound for all, or where there are top_k of it)
    if (fits && s.by_k && s.top_k > kQuota) {
      const float most = nth_bound<W>(lds.raised, 1);
      fits = most <= bound || count_from<T>(lds.joined(), n, most) >= s.top_k;
    }
  }
  if (fits) {
    if (w > 0 && n > RowLds<W>::kRanked) return;
    const u64 *list = lds.joined();
    u64 border = ~(u64)0;
    if (n <= RowLds<W>::kRanked && (s.by_k || s.by_p)) {
      // the keys in their order, and how many of them the filters keep
      for (int j = threadIdx.x; j < n; j += 64 * W) lds.sorted[rank_among(list, n, list[j])] = list[j];
      __syncthreads();
      if (w > 0) return;
      int keep = s.by_k && s.top_k < n ? s.top_k : n;
      if (s.by_p) {
        const auto power = [&](int j) { return j < keep ? e.of(logit_of<T>(lds.sorted[j])) : 0.; };
        double before = 0, of = all;
        if (s.by_k) {
          of = 0;
          for (int j = lane; j < keep; j += 64) of += power(j);
          of = wave_sum(of);
        }
        const double target = s.top_p * of;   // (the first ones that sum to it)
        int less = 0;
        for (int j = 0; j < keep; j += 64) {
          const double upto = wave_scan(power(j + lane));
          less += __builtin_popcountll(__ballot(j + lane < keep && before + upto < target));
          before += from_lane(upto, 63);
        }
        keep = less + 1 < keep ? less + 1 : keep;
      }
      border = lds.sorted[keep - 1];
    } else {
      if (w > 0) return;
      const u64 first = first_key<T>(top);
      border = last_key<T>(bound);
      if (s.by_k)
        border = find_border<true>(list, n, first, border, [](u64) { return (u64)1; }, [&](u64) { return (u64)s.top_k; }, lds.wave);
      if (s.by_p)
        border = find_border<false>(list, n, first, border, [&](u64 r) { return e.mass(logit_of<T>(r)); },
                                    [&](u64 total) { return target_of_p(s, e, total, all); }, lds.wave);
    }
    const Kept<T> kept = {border, __builtin_fmax(s.min_p, kNoPower)};
    const auto power = [&](int j) { return kept.power(e, index_of(list[j]), logit_of<T>(list[j])); };
    double t = 0;
    for (int j = lane; j < n; j += 64) t += power(j);
    const double total = wave_sum(t);
    double before;
    const int j = find_part(n, uniform_of(p, row) * total, power, before);
    if (lane == 0) write_token(p, row, s, index_of(list[j]), logit_of<T>(list[j]), top, all, total);
    return;
  }
  if constexpr (again(W)) {
    __syncthreads();
    double sum = all;
    if (!row_of.fits) {   // (some waves have not gone to their stretches' ends)
      sum = measure_row<T, 64 * W>(z, s, p, top, e, lds.part);
      if (!(__builtin_fabsf(top) < __builtin_inff())) {
        if (threadIdx.x == 0) write_bad(p, row);
        return;
      }
      bound = bound_of(want, top, top, sum, V);
    }
    sample_from_memory<T, 64 * W>(z, s, row, p, e, top, sum, bound, lds.block, &lds.chunk[0][0]);
  } else {
    if (threadIdx.x == 0) gmem(later)[row] = 1;
  }
}

// The rows that were left, in blocks of 1024 threads.
constexpr int kLaterThreads = 1024, kLaterBlocks = 512;
// f(row) for the marked rows that are this block's: the marks of THR of its rows are read at once.
template <int THR, class F>
__device__ __forceinline__ void marked_rows(const int32_t *later, int32_t rows, F f) {
  __shared__ u64 marks[THR / 64];
  const int64_t step = gridDim.x;
  for (int64_t base = blockIdx.x; base < rows; base += THR * step) {
    const int64_t row = base + threadIdx.x * step;
    const u64 mine = __ballot(row < rows && gmem(later)[row < rows ? row : 0] != 0);
    if ((threadIdx.x & 63) == 0) marks[threadIdx.x >> 6] = mine;
    __syncthreads();
    for (int w = 0; w < THR / 64; ++w)
      for (u64 m = marks[w]; m != 0; m &= m - 1) {
        f(base + (w * 64 + lane_of(m)) * step);
        __syncthreads();
      }
    __syncthreads();
  }
}
template <class T>
__global__ __launch_bounds__(kLaterThreads) void sample_later_kernel(const T *logits, SampleParams p, const int32_t *later,
                                                                     int32_t rows) {
  constexpr int THR = kLaterThreads;
  __shared__ union {
    BlockLds<THR> block;
    double chunk[HIMUON_TOP_VOCAB / (4 * 64)];
  } lds;
  __shared__ double wave[THR / 64];
  marked_rows<THR>(later, rows, [&](int64_t row) {
    const T *z = logits + row * p.ld_logits;
    const Settings s = settings_of(p, row);
    Powers e;
    e.unit = __builtin_amdgcn_ldexp(1., p.mass_bits);
    float top;
    const double all = measure_row<T, THR>(z, s, p, top, e, wave);
    __syncthreads();
    if (!(__builtin_fabsf(top) < __builtin_inff())) {
      if (threadIdx.x == 0) write_bad(p, row);
      return;
    }
    sample_from_memory<T, THR>(z, s, row, p, e, top, all, -__FLT_MAX__, lds.block, lds.chunk);
  });
}

struct TopParams {
  void *value;
  int64_t *index;
  float *rest;
  int64_t ld_logits, ld_top;
  int32_t vocab, k;
  float k2;         // log2(e) / temperature
  float inv_temp;
  double k1, temp;  // log2(e) / temperature, temperature
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
__device__ __forceinline__ void write_rest(float max, float sum, const TopParams &p, int64_t row, Softmax *waves) {
  const Softmax s = block_softmax<THR / 64>(max, sum, p.k2, waves);
  if (threadIdx.x == 0)
    gmem(p.rest)[row] = s.sum == 0.f ? -__builtin_inff() : s.ref * p.inv_temp + kLn2 * __builtin_amdgcn_logf(s.sum);
}
template <class T>
__device__ __forceinline__ void write_entry(u64 key, int i, const TopParams &p, int64_t row) {
  gmem(p.index)[row * p.ld_top + i] = index_of(key);
  Vec<T>::store1(reinterpret_cast<T *>(p.value) + row * p.ld_top + i, logit_of<T>(key));
}

// A row that is read from memory for every pass over it, by the THR threads of a block; keys: room for
// sort_size(k) of them, which may be in the histogram's place.
template <class T, int THR>
__device__ __forceinline__ void top_from_memory(const T *z, const TopParams &p, int64_t row, BlockLds<THR> &block, u64 *keys,
                                                Softmax *waves, int &found) {
  constexpr int N = Vec<T>::N;
  const int V = p.vocab, tid = threadIdx.x;
  u64 border = ~(u64)0;
  if (tid == 0) found = 0;
  if (p.k < V)
    border = find_border_in_row<T, THR, true>(z, V, 0, last_key<T>(-__builtin_inff()), [](float) { return (u64)1; },
                                              [&](u64) { return (u64)p.k; }, block);
  __syncthreads();
  float m = -__builtin_inff(), sum = 0.f;
  each_vector<T, THR>(z, V, [&](int at, float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const u64 r = rank_key<T>(x[e], at * N + e);
      if (at * N + e >= V) continue;
      if (r <= border) keys[atomicAdd(&found, 1)] = r;
      else m = __builtin_fmaxf(m, x[e]);
    }
  });
  const int size = sort_size(p.k);
  for (int i = p.k + tid; i < size; i += THR) keys[i] = ~(u64)0;
  __syncthreads();
  sort_keys<THR>(keys, size);
  for (int i = tid; i < p.k; i += THR) write_entry<T>(keys[i], i, p, row);
  const float ref = ref_of(m);
  each_vector<T, THR>(z, V, [&](int at, float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (at * N + e < V && rank_key<T>(x[e], at * N + e) > border) sum += pow2(x[e], p.k2, ref);
  });
  write_rest<THR>(m, sum, p, row, waves);
}

template <class T, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(W == 2 ? 3 : 4)))
void top_kernel(const T *logits, TopParams p, int32_t *later) {
  constexpr int THR = 64 * W;
  __shared__ RowLds<W> lds;
  __shared__ Softmax waves[W];
  const int64_t row = blockIdx.x;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, V = p.vocab, turns = turns_of<T>(V);
  const T *z = logits + row * p.ld_logits;
  const int t0 = stretch_turn(turns, w, W), t1 = stretch_turn(turns, w + 1, W);
  Turn<T> now;
  now.load(z, t0 < t1 ? t0 : turns, V);
  const int quota = p.k < kQuota ? p.k : kQuota;
  const Shares share = shares_of<W>(p.k);
  const Wants want = {quota, raise_at(quota, true), raise_at(quota, false), p.k1, p.temp, 0., 0., false};
  float top, bound;
  first_bounds<T, W>(now, share, lds, top, bound);
  const Stretch mine = sweep<T, true>(now, z, V, t0, t1, want, false, bound, bound, lds.list[w], nullptr,
                                                 turns > W && share.ranks <= W ? share.quota : 0);
  leave_stretch<W>(mine, lds);
  const Together row_of = together(lds);
  // (the others' sums, relative to the largest of their references)
  const float ref = lane < W ? lds.out[lane].ref : -__builtin_inff(), max = wave_max(row_of.sum > 0. ? ref : -__builtin_inff());
  const double sum = wave_sum(row_of.sum > 0. ? row_of.sum * pow2_exact(((double)ref - max) * p.k1) : 0.);
  // (where the others are so far below that their powers lose bits, they are taken from their own largest)
  bool fits = row_of.fits && __builtin_fabsf(row_of.top) < __builtin_inff() && row_of.listed >= p.k &&
              (row_of.listed == V || sum >= 0x1p-60);
  if (fits) {
    bound = share.ranks <= W ? nth_bound<W>(lds.last_bound, share.ranks) : -__FLT_MAX__;
    // (what is below the bound is one of the others)
    float m = sum > 0. ? max : -__builtin_inff();
    const int own = lds.out[w].n;
    const u64 *list = lds.list[w];
    for (int j = lane; j < own; j += 64) {
      const float x = logit_of<T>(list[j]);
      if (x < bound) m = __builtin_fmaxf(m, x);
    }
    float rest = 0.f;   // of those, relative to m (they are before one wave's list is shortened)
    {
      const float to = ref_of(m);
      for (int j = lane; j < own; j += 64) {
        const float x = logit_of<T>(list[j]);
        if (x < bound) rest += pow2(x, p.k2, to);
      }
      if (threadIdx.x == 0 && sum > 0.) rest += (float)sum * pow2(max, p.k2, to);
    }
    wave_sync();
    const int n = join_lists<T>(lds, bound);
    u64 *keys = lds.joined();
    fits = n <= RowLds<W>::kJoined && n >= p.k;
    // (where a stretch's list followed its kQuota-th largest, the lists hold what is not below what that raised its bound
    // to: enough where that is not above the bound for all, or where there are k of it)
    if (fits && p.k > kQuota) {
      const float most = nth_bound<W>(lds.raised, 1);
      fits = most <= bound || count_from<T>(keys, n, most) >= p.k;
    }
    if (fits) {
      const auto other = [&](u64 r) {
        const float x = logit_of<T>(r), to = __builtin_fmaxf(m, x);
        rest = (rest > 0.f ? rest * pow2(m, p.k2, ref_of(to)) : 0.f) + pow2(x, p.k2, ref_of(to));
        m = to;
      };
      if (n <= RowLds<W>::kRanked) {
        for (int j = threadIdx.x; j < n; j += THR) {
          const u64 r = keys[j];
          const int rank = rank_among(keys, n, r);
          if (rank < p.k) write_entry<T>(r, rank, p, row);
          else other(r);
        }
      } else {
        const int size = sort_size(n);
        for (int i = n + threadIdx.x; i < size; i += THR) keys[i] = ~(u64)0;
        __syncthreads();
        sort_keys<THR>(keys, size);
        for (int j = threadIdx.x; j < n; j += THR) {
          if (j < p.k) write_entry<T>(keys[j], j, p, row);
          else other(keys[j]);
        }
      }
      write_rest<THR>(m, rest, p, row, waves);
    }
  }
  if constexpr (again(W)) {
    if (fits) return;
    __syncthreads();
    top_from_memory<T, THR>(z, p, row, lds.block, lds.joined(), waves, lds.count[0]);
  } else {
    if (threadIdx.x == 0) gmem(later)[row] = !fits;
  }
}

template <class T>
__global__ __launch_bounds__(kLaterThreads) void top_later_kernel(const T *logits, TopParams p, const int32_t *later,
                                                                  int32_t rows) {
  constexpr int THR = kLaterThreads;
  __shared__ BlockLds<THR> block;
  __shared__ u64 keys[HIMUON_TOP_MOST];
  __shared__ Softmax waves[THR / 64];
  __shared__ int found;
  marked_rows<THR>(later, rows, [&](int64_t row) {
    top_from_memory<T, THR>(logits + row * p.ld_logits, p, row, block, keys, waves, found);
  });
}

constexpr int64_t kLaunchRows = (int64_t)1 << 21;   // a grid holds fewer than 2^32 threads

// Waves for a row: enough of them to fill the chip (256 CUs with 16 each: draws of 1024 x 128256 bf16 take 115 us with 4
// waves a row, 122 with 2 and 180 with 1; the top 100 of 1023 x 50257 fp32 82 us with 8, 89 with 4 and 127 with 16), and as
// many as its stretches' lengths ask for.  A block of 16 waves has a CU for itself, so 16 only where all blocks run at once
// (500 x 50257 fp32, top_p: 44.5 us with 8, 52.6 with 16).
constexpr int kFillWaves = 4096;
// The k up to which W waves take a row.  Top k of 4096 rows, us:
//                            k =    64   150   180   216   224   300   440   640   700  1024
//   128256 bf16 tokens, 1 wave     295   367   580   522   697  1528  1578  1689  1708  1800
//                       2 waves    416   520   558   626   641   710  1148  1704  1721  1814
//                       4 waves    376   470   494   560   574   641   682  1024  1723  1483
//                       8 waves    387   441   469   514   513   650   802   943  1022  1126
//   50257 fp32 tokens,  1 wave     220   283         343         804         902         929
//                       4 waves    264   350         424         506         771         742
//                       8 waves    281   323         373         482         769         917
// One wave leads up to 150 and with fp32 to 216 (in between it depends on how often its list's bound is raised); 4 waves
// follow as long as their joined list of 1024 keys has room, which ends between 640 and 700.
constexpr int most_of(int W) { return W >= 8 ? HIMUON_TOP_MOST : W == 4 ? 640 : 216; }
int waves_of(int64_t rows, int64_t vecs, int least) {
  const int64_t turns = (vecs + kTurn - 1) / kTurn;
  int W = 1;
  while (W < 16 && (W < least || turns > (int64_t)W * kTurns || (rows * W < (W < 8 ? kFillWaves : kFillWaves / 2) && W < turns))) W *= 2;
  return W;
}
template <class F>
void with_waves(int W, F f) {
  if (W == 1) f(std::integral_constant<int, 1>());
  else if (W == 2) f(std::integral_constant<int, 2>());
  else if (W == 4) f(std::integral_constant<int, 4>());
  else if (W == 8) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
}

template <class T>
hipError_t launch_sample_t(const himuon_sampling &c, SampleParams p, int32_t *later, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  // (a stretch's list holds its kQuota largest for certain; settings of each row are not known here; what top_p alone
  // keeps often takes more than a list or two: 4096 x 128256 bf16, 0.9: 522 us with 4 waves, 724 with 2, 918 with 1.
  // Rows that keep more than the lists hold are read again: a top_k of a row's own from some 700 on with 4 waves (4096 x
  // 128256 bf16: 934 us for 641, 1790 for 880), one for all rows above 1024 with 8 (1057 us for 1024, 2049 for 1500))
  const bool by_p = c.row_top_p || c.top_p < 1.;
  int least = c.row_top_k || (by_p && !c.top_k) ? 4 : 1;
  while (!c.row_top_k && least < 8 && most_of(least) < c.top_k) least *= 2;
  // (without filters, temperature 0 among them, no row has a list)
  const bool lists = c.row_top_k || c.top_k || by_p || c.row_min_p || c.min_p > 0. || c.row_temperature || c.temperature == 0.;
  const int W = waves_of(c.rows, (c.vocab + Vec<T>::N - 1) / Vec<T>::N, least);
  for (int64_t r = 0; r < c.rows; r += kLaunchRows) {
    const unsigned rows = (unsigned)(c.rows - r < kLaunchRows ? c.rows - r : kLaunchRows);
    with_waves(W, [&](auto waves) {
      constexpr int kWaves = decltype(waves)::value;
      hipLaunchKernelGGL((sample_kernel<T, kWaves>), dim3(rows), dim3(64 * kWaves), 0, stream, z + r * c.ld_logits, p, later);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!again(W) && lists) {
      hipLaunchKernelGGL((sample_later_kernel<T>), dim3(rows < kLaterBlocks ? rows : kLaterBlocks), dim3(kLaterThreads), 0,
                         stream, z + r * c.ld_logits, p, later, (int32_t)rows);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      later += rows;
    }
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
hipError_t launch_top_t(const himuon_top &c, TopParams p, int32_t *later, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  int least = 1;
  while (most_of(least) < c.k) least *= 2;
  const int W = waves_of(c.rows, (c.vocab + Vec<T>::N - 1) / Vec<T>::N, least);
  for (int64_t r = 0; r < c.rows; r += kLaunchRows) {
    const unsigned rows = (unsigned)(c.rows - r < kLaunchRows ? c.rows - r : kLaunchRows);
    with_waves(W, [&](auto waves) {
      constexpr int kWaves = decltype(waves)::value;
      hipLaunchKernelGGL((top_kernel<T, kWaves>), dim3(rows), dim3(64 * kWaves), 0, stream, z + r * c.ld_logits, p, later);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!again(W)) {
      hipLaunchKernelGGL((top_later_kernel<T>), dim3(rows < kLaterBlocks ? rows : kLaterBlocks), dim3(kLaterThreads), 0,
                         stream, z + r * c.ld_logits, p, later, (int32_t)rows);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      later += rows;
    }
    p.value = reinterpret_cast<T *>(p.value) + rows * p.ld_top;
    p.index += rows * p.ld_top;
    p.rest += rows;
  }
  return hipSuccess;
}

}  // namespace

// A mark for each row that the first launch may leave to the second.
size_t sample_workspace(const himuon_sampling &c) { return (size_t)(c.rows + 1) / 2 * 8; }
size_t top_workspace(const himuon_top &c) { return (size_t)(c.rows + 1) / 2 * 8; }

hipError_t launch_sample(const himuon_sampling &c, void *workspace, hipStream_t stream) {
  SampleParams p{};
  int32_t *later = reinterpret_cast<int32_t *>(workspace);
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
  return c.dtype == HIMUON_BF16 ? launch_sample_t<__bf16>(c, p, later, stream) : launch_sample_t<float>(c, p, later, stream);
}

hipError_t launch_top(const himuon_top &c, void *workspace, hipStream_t stream) {
  TopParams p{};
  int32_t *later = reinterpret_cast<int32_t *>(workspace);
  p.value = c.value;
  p.index = c.index;
  p.rest = c.rest;
  p.ld_logits = c.ld_logits;
  p.ld_top = c.ld_top;
  p.vocab = (int32_t)c.vocab;
  p.k = c.k;
  p.k2 = (float)(kLog2e / c.temperature);
  p.inv_temp = (float)(1. / c.temperature);
  p.k1 = kLog2e / c.temperature;
  p.temp = c.temperature;
  return c.dtype == HIMUON_BF16 ? launch_top_t<__bf16>(c, p, later, stream) : launch_top_t<float>(c, p, later, stream);
}

}  // namespace himuon
