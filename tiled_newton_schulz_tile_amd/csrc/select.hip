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
// A border and a draw decide about whole tokens, and a sum in fp32 that is off by 1e-7 decides
// wrongly in one row of a hundred where 1e5 tokens share the probability.  Powers are therefore
// taken in fp64 (fp64 multiply-adds run at the rate of fp32 ones here), sums of probabilities that
// go through atomics are whole multiples of a power of two in 64 bits, and all others have a fixed
// order: results do not depend on timing.
#include "device_common.h"
#include "himuon_internal.h"
#include "row_softmax.h"

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

// Calls f(index, logit) for every element of a row, all threads of the block in step.
template <class T, int THR>
struct RowSource {
  const T *z;
  int V;
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    constexpr int N = Vec<T>::N;
    const int vecs = V / N;
    for (int at = threadIdx.x; at < vecs; at += THR) {
      float x[N];
      Vec<T>::unpack(Vec<T>::load(z + (int64_t)at * N), x);
#pragma unroll
      for (int e = 0; e < N; ++e) f(at * N + e, x[e]);
    }
    const int rest = vecs * N + threadIdx.x;
    if (rest < V) f(rest, Vec<T>::load1(z + rest));
  }
};

constexpr int kBins = 1024;
struct SelectLds {
  u64 mass[kBins];      // what a bin weighs
  unsigned count[kBins];
  u64 wave[16];
  u64 before;           // the weight before the bin that was found
  int bin;              // -1: none
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
// one that reaches it.  weight(z): an element's weight (the target at most 2^64 - 1 in all).  Where
// all weigh less: last.  target(total): the target, given what all weigh together.
template <int THR, class SOURCE, class WEIGHT, class TARGET>
__device__ __forceinline__ u64 find_border(const SOURCE &src, u64 first, u64 last, WEIGHT weight, TARGET target_of,
                                           SelectLds &lds) {
  constexpr int B = kBins / THR > 0 ? kBins / THR : 1;   // bins a thread
  u64 base = 0, target = 0;
  const u64 end = last;
  for (bool top = true;; top = false) {
    const int bits = 64 - __builtin_clzll((last - first) | 1);
    const int shift = bits > 10 ? bits - 10 : 0;
#pragma unroll
    for (int i = 0; i < kBins; i += THR)
      if (i + (int)threadIdx.x < kBins) {
        lds.mass[i + threadIdx.x] = 0;
        lds.count[i + threadIdx.x] = 0;
      }
    if (threadIdx.x == 0) lds.bin = -1;
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
    if (top) {
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
    if (lds.bin < 0) return end;   // (a target of 0)
    base = lds.before;
    first += (u64)lds.bin << shift;
    last = last - first < ((u64)1 << shift) - 1 ? last : first + (((u64)1 << shift) - 1);
    const bool done = shift == 0 || lds.count[lds.bin] == 1;
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

// One block per row, which it reads from memory for every pass over it.
template <class T, int THR>
__global__ __launch_bounds__(THR) void sample_kernel(const T *logits, SampleParams p) {
  constexpr int N = Vec<T>::N;
  extern __shared__ double chunk[];   // what each wave's vectors of a turn over the row weigh
  __shared__ SelectLds lds;
  __shared__ double wave[16];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, V = p.vocab, vecs = V / N;
  const T *z = logits + row * p.ld_logits;
  const RowSource<T, THR> src = {z, V};
  const double temp = p.temperature ? (double)gmem(p.temperature)[row] : p.T;
  const bool greedy = temp == 0.;
  const bool good = greedy || (temp >= 0x1p-20 && temp <= 0x1p20);
  const double top_p = p.top_p ? (double)gmem(p.top_p)[row] : p.p, min_p = p.min_p ? (double)gmem(p.min_p)[row] : p.m;
  int top_k = greedy ? 1 : p.top_k ? gmem(p.top_k)[row] : p.k;
  if (top_k <= 0 || top_k > V) top_k = V;
  const double k = kLog2e / (good && !greedy ? temp : 1.);

  float m = -__builtin_inff();
  src.each([&](int, float x) { m = __builtin_fmaxf(m, x); });
  m = wave_max(m);
  if (lane == 0) wave[tid >> 6] = m;
  __syncthreads();
  float top = -__builtin_inff();
#pragma unroll
  for (int w = 0; w < THR / 64; ++w) top = __builtin_fmaxf(top, (float)wave[w]);
  double mine = 0;
  src.each([&](int, float x) { mine += pow2_exact(((double)x - top) * k); });
  const double all = block_sum_in_order<THR>(mine, wave);
  if (!(all > 0.) || !good) {   // NaN or +inf in the row, nothing but -inf, no such temperature
    if (tid == 0) {
      gmem(p.token)[row] = -1;
      gmem(p.logp)[row] = gmem(p.kept)[row] = __builtin_nanf("");
    }
    return;
  }

  const double unit = __builtin_amdgcn_ldexp(1., p.mass_bits);
  const auto mass = [&](float x) { return (u64)(pow2_exact(((double)x - top) * k) * unit + 0.5); };
  u64 border = ~(u64)0;
  const u64 first = (u64)down_key(top) << 32, last = (u64)down_key(-__FLT_MAX__) << 32 | 0xffffffffu;
  if (top_k < V)
    border = find_border<THR>(src, first, last, [](float) { return (u64)1; }, [&](u64) { return (u64)top_k; }, lds);
  if (!greedy && top_p < 1.) {
    const u64 to = border < last ? border : last;
    border = find_border<THR>(src, first, to, mass, [&](u64 total) {
      const double t = __builtin_ceil((top_p > 0. ? top_p : 0.) * (double)total);
      return t < 1. ? (u64)1 : (u64)t;
    }, lds);
  }
  const double least = !greedy && min_p > 0. ? (min_p < 1. ? min_p : 1.) : 0.;
  const auto weight = [&](int index, float x) {
    const double e = pow2_exact(((double)x - top) * k);
    return x > -__builtin_inff() && rank_key(x, index) <= border && e >= least ? e : 0.;
  };

  // the draw: a wave's 64 vectors of a turn are consecutive elements, so the chunks are in order
  const int turns = (vecs + THR - 1) / THR, chunks = turns * (THR / 64) + 1;
  for (int t = 0; t < turns; ++t) {
    const int at = t * THR + tid;
    double s = 0;
    if (at < vecs) {
      float x[N];
      Vec<T>::unpack(Vec<T>::load(z + (int64_t)at * N), x);
#pragma unroll
      for (int e = 0; e < N; ++e) s += weight(at * N + e, x[e]);
    }
    s = wave_sum(s);
    if (lane == 0) chunk[t * (THR / 64) + (tid >> 6)] = s;
  }
  if (tid < 64) {
    const int rest = vecs * N + lane;
    const double s = wave_sum(rest < V ? weight(rest, Vec<T>::load1(z + rest)) : 0.);
    if (lane == 0) chunk[chunks - 1] = s;
  }
  __syncthreads();
  if (tid >= 64) return;
  // one wave: the chunk in which the sum passes the target, then the lane, then the element
  double sum = 0;
  for (int c = lane; c < chunks; c += 64) sum += chunk[c];
  const double total = wave_sum(sum);
  double u = (double)gmem(p.uniform)[row];
  u = u > 0. ? (u < 1. ? u : 1.) : 0.;   // (NaN is 0)
  const double target = u * total;
  double before = 0;
  int at = -1, last_some = 0;
  double at_before = 0, some_before = 0;
  for (int c0 = 0; c0 < chunks && at < 0; c0 += 64) {
    const double w = c0 + lane < chunks ? chunk[c0 + lane] : 0.;
    double s = w;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double up = __shfl_up(s, d);
      if (lane >= d) s += up;
    }
    const u64 hit = __ballot(w > 0. && before + s > target), some = __ballot(w > 0.);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      at = c0 + l;
      at_before = l ? before + __shfl(s, l - 1) : before;
    } else if (some) {
      const int l = 63 - __builtin_clzll(some);
      last_some = c0 + l;
      some_before = l ? before + __shfl(s, l - 1) : before;
    }
    before += __shfl(s, 63);
  }
  if (at < 0) {   // the target is the whole sum: the last token that is kept
    at = last_some;
    at_before = some_before;
  }
  const bool rest = at == chunks - 1;
  const int i0 = rest ? vecs * N + lane : ((at / (THR / 64)) * THR + (at % (THR / 64)) * 64 + lane) * N;
  double w[N];
  float x[N];
  double own = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const bool in = rest ? e == 0 && i0 < V : i0 + e < vecs * N;
    x[e] = in ? Vec<T>::load1(z + i0 + e) : -__builtin_inff();
    w[e] = in ? weight(i0 + e, x[e]) : 0.;
    own += w[e];
  }
  double s = own;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double up = __shfl_up(s, d);
    if (lane >= d) s += up;
  }
  const u64 hit = __ballot(own > 0. && at_before + s > target), some = __ballot(own > 0.);
  const int l = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some);
  if (lane != l) return;
  double run = at_before + s - own;
  int token = -1;
  float logit = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (w[e] > 0. && (token < 0 || run <= target)) {
      token = i0 + e;
      logit = x[e];
    }
    run += w[e];
  }
  gmem(p.token)[row] = token;
  gmem(p.logp)[row] = greedy ? 0.f : (float)(((double)logit - top) * (1. / temp) - log(all));
  gmem(p.kept)[row] = greedy ? 1.f : (float)(total / all);
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

template <class T, int THR>
__global__ __launch_bounds__(THR) void top_kernel(const T *logits, TopParams p) {
  __shared__ SelectLds lds;
  __shared__ u64 list[HIMUON_TOP_MOST];
  __shared__ Softmax waves[16];
  __shared__ int n;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, V = p.vocab;
  const T *z = logits + row * p.ld_logits;
  const RowSource<T, THR> src = {z, V};
  u64 border = ~(u64)0;
  if (p.k < V)
    border = find_border<THR>(src, 0, ~(u64)0, [](float) { return (u64)1; }, [&](u64) { return (u64)p.k; }, lds);
  int pow2k = 64;
  while (pow2k < p.k) pow2k *= 2;
  for (int i = tid; i < pow2k; i += THR) list[i] = ~(u64)0;
  if (tid == 0) n = 0;
  __syncthreads();
  float m = -__builtin_inff();
  src.each([&](int index, float x) {
    const u64 r = rank_key(x, index);
    if (r <= border) list[atomicAdd(&n, 1)] = r;
    else m = __builtin_fmaxf(m, x);
  });
  __syncthreads();
  for (int size = 2; size <= pow2k; size *= 2)
    for (int step = size / 2; step > 0; step /= 2) {
      for (int i = tid; i < pow2k / 2; i += THR) {
        const int a = i / step * (2 * step) + i % step, b = a + step;
        const bool up = !(a & size);
        const u64 x = list[a], y = list[b];
        if ((x > y) == up) {
          list[a] = y;
          list[b] = x;
        }
      }
      __syncthreads();
    }
  for (int i = tid; i < p.k; i += THR) {
    const int index = (int)(unsigned)list[i];
    gmem(p.index)[row * p.ld_top + i] = index;
    const T x = *gmem(z + index);
    *gmem(reinterpret_cast<T *>(p.value) + row * p.ld_top + i) = x;
  }
  // the others, from their largest
  float sum = 0.f;
  const float ref = ref_of(m);
  src.each([&](int index, float x) {
    if (rank_key(x, index) > border) sum += pow2(x, p.k2, ref);
  });
  const Softmax s = block_softmax<THR / 64>(m, sum, p.k2, waves);
  if (tid == 0)
    gmem(p.rest)[row] = s.sum == 0.f ? -__builtin_inff() : s.ref * p.inv_temp + kLn2 * __builtin_amdgcn_logf(s.sum);
}

constexpr int64_t kLaunchRows = (int64_t)1 << 21;   // a grid holds fewer than 2^32 threads

template <class T, int THR>
void launch_sample_rows(const T *z, unsigned rows, const SampleParams &p, hipStream_t stream) {
  const int64_t vecs = p.vocab / Vec<T>::N;
  const size_t lds = ((vecs + THR - 1) / THR * (THR / 64) + 1) * sizeof(double);
  hipLaunchKernelGGL((sample_kernel<T, THR>), dim3(rows), dim3(THR), lds, stream, z, p);
}
template <class T>
hipError_t launch_sample_t(const himuon_sampling &c, SampleParams p, hipStream_t stream) {
  const T *z = reinterpret_cast<const T *>(c.logits);
  for (int64_t r = 0; r < c.rows; r += kLaunchRows) {
    const unsigned rows = (unsigned)(c.rows - r < kLaunchRows ? c.rows - r : kLaunchRows);
    if (c.vocab <= 8192) launch_sample_rows<T, 256>(z + r * c.ld_logits, rows, p, stream);
    else launch_sample_rows<T, 1024>(z + r * c.ld_logits, rows, p, stream);
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
  for (int64_t r = 0; r < c.rows; r += kLaunchRows) {
    const unsigned rows = (unsigned)(c.rows - r < kLaunchRows ? c.rows - r : kLaunchRows);
    if (c.vocab <= 8192) hipLaunchKernelGGL((top_kernel<T, 256>), dim3(rows), dim3(256), 0, stream, z + r * c.ld_logits, p);
    else hipLaunchKernelGGL((top_kernel<T, 1024>), dim3(rows), dim3(1024), 0, stream, z + r * c.ld_logits, p);
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
