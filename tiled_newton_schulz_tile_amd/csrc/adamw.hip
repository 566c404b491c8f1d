// AdamW over many tensors in one launch, with fp32 or 8-bit states, and the norm of many
// gradients.  Both are streams: every element of every tensor crosses HBM once.
//
// The tensors' descriptors travel in the kernel arguments while they fit (so a call needs
// no table in device memory, no upload and no wait, and pointers may change from step to
// step), or in a table in device memory that the caller uploads once.  Every tensor is cut
// into chunks of 1024 elements; a block finds the tensor of its chunk with one load
// per lane of the first-chunk table and a ballot.
//
// Tensors may start at any element (views of a flattened bucket do): vectors are declared
// with the alignment of one element and the hardware takes unaligned global accesses.
#include "device_common.h"
#include "himuon_internal.h"
#include "wave_reduce.h"

#include <cmath>

namespace himuon {
namespace {

using namespace dev;

constexpr int THREADS = 256;

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned short u16x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned short u16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef unsigned u32u __attribute__((aligned(1)));

__device__ __forceinline__ float load1(const float *p, int64_t i) { return gmem(p)[i]; }
__device__ __forceinline__ float load1(const __bf16 *p, int64_t i) {
  return bf16_bits_to_f32(gmem(reinterpret_cast<const unsigned short *>(p))[i]);
}
__device__ __forceinline__ void store1(float *p, int64_t i, float x) { gmem(p)[i] = x; }
__device__ __forceinline__ void store1(__bf16 *p, int64_t i, float x) {
  gmem(reinterpret_cast<unsigned short *>(p))[i] = to_bf16_bits(x);
}
// NT: past the caches (non-temporal).  (Not through a template on the vector type: deduction
// would drop its alignment.)
template <bool NT>
__device__ __forceinline__ f32x4 load4(const float *p, int64_t i) {
  const GLOBAL_AS f32x4u *q = reinterpret_cast<const GLOBAL_AS f32x4u *>(gmem(p + i));
  if constexpr (NT) return __builtin_nontemporal_load(q);
  return *q;
}
template <bool NT>
__device__ __forceinline__ f32x4 load4(const __bf16 *p, int64_t i) {
  const GLOBAL_AS u16x4u *q = reinterpret_cast<const GLOBAL_AS u16x4u *>(gmem(p + i));
  u16x4 h;
  if constexpr (NT) h = __builtin_nontemporal_load(q);
  else h = *q;
  return f32x4{bf16_bits_to_f32(h[0]), bf16_bits_to_f32(h[1]), bf16_bits_to_f32(h[2]), bf16_bits_to_f32(h[3])};
}
template <bool NT>
__device__ __forceinline__ void store4(float *p, int64_t i, f32x4 x) {
  GLOBAL_AS f32x4u *q = reinterpret_cast<GLOBAL_AS f32x4u *>(gmem(p + i));
  if constexpr (NT) __builtin_nontemporal_store(x, q);
  else *q = x;
}
template <bool NT>
__device__ __forceinline__ void store4(__bf16 *p, int64_t i, f32x4 x) {
  GLOBAL_AS u16x4u *q = reinterpret_cast<GLOBAL_AS u16x4u *>(gmem(p + i));
  const u16x4 h = {to_bf16_bits(x[0]), to_bf16_bits(x[1]), to_bf16_bits(x[2]), to_bf16_bits(x[3])};
  if constexpr (NT) __builtin_nontemporal_store(h, q);
  else *q = h;
}
// n (0..4) elements from i on; what lies beyond them reads as zero and is not written
template <bool NT, class T>
__device__ __forceinline__ f32x4 load_upto4(const T *p, int64_t i, int n) {
  if (n >= 4) return load4<NT>(p, i);
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) x[e] = load1(p, i + e);
  return x;
}
template <bool NT, class T>
__device__ __forceinline__ void store_upto4(T *p, int64_t i, int n, f32x4 x) {
  if (n >= 4) return store4<NT>(p, i, x);
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) store1(p, i + e, x[e]);
}

// ------------------------------------------------------------------ tables in arguments
// One tensor.  8-bit entries hold two scale pointers more.
template <int BITS>
struct Entry {
  void *w;
  const void *g;
  void *m, *v;
  int64_t n;
  float weight_decay;
};
template <>
struct Entry<8> {
  void *w;
  const void *g;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  float weight_decay;
};
// Up to kMost tensors travel in the arguments, which have 4 KB; a call of kFew at most takes a
// small table, for the launch of the large one costs the host a microsecond and a half more.
template <int BITS>
constexpr int kMost = BITS == 8 ? 56 : 72;
constexpr int kFew = 8;

template <int BITS, int CAP>
struct ArgTable {
  int32_t n;
  int32_t first[CAP + 1];   // first chunk of each tensor; [n]: all chunks
  Entry<BITS> t[CAP];
  __device__ __forceinline__ const int32_t *firsts() const { return first; }
  __device__ __forceinline__ const Entry<BITS> *entries() const { return t; }
};
static_assert(sizeof(ArgTable<32, kMost<32>>) + sizeof(AdamWParams) <= 4096, "kernel arguments");
static_assert(sizeof(ArgTable<8, kMost<8>>) + sizeof(AdamWParams) <= 4096, "kernel arguments");

// The same in device memory: n + 1 first chunks, then the entries at entry_offset(n).
size_t entry_offset(int64_t n) { return ((size_t)(n + 1) * sizeof(int32_t) + 15) / 16 * 16; }
template <int BITS>
struct DeviceTable {
  int32_t n;
  const int32_t *first;
  const Entry<BITS> *t;
  __device__ __forceinline__ const int32_t *firsts() const { return first; }
  __device__ __forceinline__ const Entry<BITS> *entries() const { return t; }
};

constexpr int kNormTensors = 198;
struct NormTable {
  int32_t n, shift;
  int32_t first[kNormTensors + 1];
  int64_t size[kNormTensors];
  const void *g[kNormTensors];
};
static_assert(sizeof(NormTable) + 64 <= 4096, "kernel arguments");

// A chunk is one vector of four elements a thread: every load of a block is in flight at once
// and nothing loops.  Chunks of 4096 took 3 % (fp32 states) and 6 % (8-bit) longer on 262 M
// elements, and leave CUs idle in a call of a few hundred thousand.
constexpr int kChunkShift = 10;
static_assert(1 << kChunkShift == 4 * THREADS, "four elements a thread");

// The tensor that chunk c belongs to: the last one whose first chunk is <= c.  (Tensors
// without elements are not in the table.)
__device__ __forceinline__ int tensor_of(const int32_t *first, int n, int c) {
  const int lane = threadIdx.x & 63;
  int count = 0;
  for (int k = 0; k < n; k += 64) {
    const bool le = k + lane < n && first[k + lane] <= c;
    count += __builtin_popcountll(__ballot(le));
  }
  return __builtin_amdgcn_readfirstlane(count - 1);
}

// ------------------------------------------------------------------ AdamW
// The weight after a step with the new first moment and the root of the new second one.  The
// hardware's reciprocal is within an ulp, far inside what the step needs, and its argument is
// eps at least, a normal number.  (The hardware's root takes subnormals for zero, and so would
// let a tiny eps divide: the rounded root is used.)
__device__ __forceinline__ float new_weight(float w, float m, float root, float decay, const AdamWParams &p) {
  const float den = __builtin_fmaf(root, p.root_scale, p.eps);
  return __builtin_fmaf(w, decay, -p.step * (m * __builtin_amdgcn_rcpf(den)));
}

template <typename W, typename G, bool NT, class TABLE>
__global__ __launch_bounds__(THREADS) void adamw32_kernel(TABLE tab, AdamWParams p) {
  const float scale = p.grad_scale ? *gmem(p.grad_scale) : 1.f;
  const int c = p.first_chunk + blockIdx.x, ti = tensor_of(tab.firsts(), tab.n, c);
  const Entry<32> &t = tab.entries()[ti];
  W *w = reinterpret_cast<W *>(t.w);
  const G *g = reinterpret_cast<const G *>(t.g);
  float *m = reinterpret_cast<float *>(t.m), *v = reinterpret_cast<float *>(t.v);
  const float decay = 1.f - p.lr * t.weight_decay;
  const int64_t i = ((int64_t)(c - tab.firsts()[ti]) << kChunkShift) + 4 * threadIdx.x;
  if (i >= t.n) return;
  const int n = t.n - i < 4 ? (int)(t.n - i) : 4;
  const f32x4 gv = load_upto4<NT>(g, i, n);
  f32x4 mv = load_upto4<NT>(m, i, n), vv = load_upto4<NT>(v, i, n), wv = load_upto4<NT>(w, i, n);
  if (scale != scale) return;   // the gradient was not finite: nothing changes
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = gv[e] * scale;
    mv[e] = __builtin_fmaf(p.beta1, mv[e], p.omb1 * x);
    vv[e] = __builtin_fmaf(p.beta2, vv[e], p.omb2 * x * x);
    wv[e] = new_weight(wv[e], mv[e], __builtin_sqrtf(vv[e]), decay, p);
  }
  store_upto4<NT>(m, i, n, mv);
  store_upto4<NT>(v, i, n, vv);
  store_upto4<NT>(w, i, n, wv);
}

// ---- 8-bit states
// A dithered rounding turns over at one of 2^16 points per gap, and a last-place difference
// carries one code in a million across such a point, which the next step's scale may show as
// a difference of a whole gap.  So the moments and codes are defined in fp32 with every
// operation rounded on its own, in the order written here (no fused multiply-adds, the root
// and the reciprocal correctly rounded): any other computation in that order gives the same
// bits.  262 M elements, fp32 weights, bf16 gradients: 590 us (6.2 TB/s), near both bounds (HBM,
// and 283 VALU instructions a block of 256, 310 with bf16 weights).
constexpr int kBlock = HIMUON_ADAMW_BLOCK;
static_assert(kBlock == 4 * 64, "a wave holds one block");
constexpr unsigned kStepM = 0x9E3779B1u, kStepR = 0x85EBCA6Bu;   // of the dither sequences

__device__ __forceinline__ f32x4 unpack_e4m3x4(unsigned x) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, true);
  return f32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ unsigned word_of(float x) { return __builtin_bit_cast(unsigned, x); }

// Largest magnitude of a wave's values, compared as bit patterns, so that a NaN is larger than
// everything and stays.
template <bool ROOT>
__device__ __forceinline__ float wave_peak(f32x4 x) {
  unsigned k = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) k = max(k, word_of(x[e]) & (ROOT ? 0xffffffffu : 0x7fffffffu));   // (word_of takes
  return __builtin_bit_cast(float, wave_max(k));   // a copy: a bit cast of x[e] itself would be that of x[0])
}
// The e4m3 code of x in units of the block's scale, rounded to a neighbouring value as the
// dither says.  y 2^-120 is an fp32 number whose exponent field, three mantissa bits on, is the
// e4m3 code of y: fp32's subnormals (which the kernel's float mode keeps) start at 2^-126 as
// e4m3's do at 2^-6, with 20 bits more.  A dither of 16 bits and a half, added at the top of the 20 bits that are cut, carries up with
// the probability of the distance to the lower neighbour.
// ROOT: x is a root, not negative; one that is not zero gets the smallest code at least.
template <bool ROOT>
__device__ __forceinline__ unsigned dithered(float x, float inv, unsigned seq) {
  const float y = __builtin_fabsf(x) * inv;
  const int code = (int)((word_of(y * 0x1p-120f) + ((seq >> 16) << 4) + 8u) >> 20);   // 126 is 448
  if constexpr (ROOT) return (unsigned)min(max(code, (int)min(word_of(x), 1u)), 126);
  return (unsigned)min(code, 126) | (word_of(x) >> 24 & 0x80u);
}
// The codes of four consecutive elements; inv = 448 / peak, 0 for a block that is held as zeros.
template <bool ROOT>
__device__ __forceinline__ unsigned codes_of(f32x4 x, float inv, unsigned seq, unsigned step) {
  unsigned word = 0;
#pragma unroll
  for (int e = 3; e >= 0; --e) word = word << 8 | dithered<ROOT>(x[e], inv, seq + e * step);
  return inv > 0.f ? word : 0u;   // (uniform over the wave)
}
// Elements that are not finite become zeros here, so that the block's others keep their scale;
// the result holds the NaN code in their places.
__device__ __forceinline__ unsigned take_out_not_finite(f32x4 &x) {
  unsigned word = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (!(__builtin_fabsf(x[e]) < __builtin_inff())) {
      x[e] = 0.f;
      word |= 0x7fu << (8 * e);
    }
  return word;
}
// 448 / peak for both moments of a wave's block, as the rounded reciprocal times 448: one
// division for the two, on even lanes the one and on odd lanes the other.
__device__ __forceinline__ void inverses(float m_peak, float r_peak, float &m_inv, float &r_inv) {
#pragma clang fp contract(off)
  const float peak = threadIdx.x & 1 ? r_peak : m_peak;
  const float inv = peak >= 0x1p-100f ? 1.f / peak * 448.f : 0.f;
  m_inv = __builtin_bit_cast(float, __builtin_amdgcn_readlane((int)word_of(inv), 0));
  r_inv = __builtin_bit_cast(float, __builtin_amdgcn_readlane((int)word_of(inv), 1));
}

// sqrt(v) rounded to nearest, for v = 0 or v in [2^-96, inf): the hardware's root s is within an ulp,
// and v against s (s - ulp) and s (s + ulp), which lie on the midpoints' squares but for a
// quarter of an ulp^2, says whether a neighbour is nearer.
__device__ __forceinline__ float rounded_sqrt(float v) {
  const float s = __builtin_amdgcn_sqrtf(v);
  const float below = __builtin_bit_cast(float, word_of(s) - 1u), above = __builtin_bit_cast(float, word_of(s) + 1u);
  float r = __builtin_fmaf(-below, s, v) <= 0.f ? below : s;
  return __builtin_fmaf(-above, s, v) > 0.f ? above : r;
}

// The root of a second moment that overflows though what it is made of does not (|g| above some
// 5e20 at beta2 0.999): from the terms times 2^-66, whose squares stay below 2^124.  The state
// holds the root, so nothing is lost; it is fp32's largest number where it rounds past that.
__device__ __forceinline__ float root_of_large(float r0, float x, const AdamWParams &p) {
#pragma clang fp contract(off)
  const float r = r0 * 0x1p-66f, g = x * 0x1p-66f;
  const float v = p.beta2 * (r * r) + p.omb2 * g * g;
  return v < __builtin_inff() ? __builtin_fminf(__builtin_sqrtf(v) * 0x1p66f, 0x1.fffffep127f) : v;
}

__device__ __forceinline__ unsigned load_codes(const unsigned char *p, int64_t i, int n) {
  if (n >= 4) return *reinterpret_cast<const GLOBAL_AS u32u *>(gmem(p + i));
  unsigned word = 0;
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) word |= (unsigned)gmem(p)[i + e] << (8 * e);
  return word;
}
__device__ __forceinline__ void store_codes(unsigned char *p, int64_t i, int n, unsigned word) {
  if (n >= 4) {
    *reinterpret_cast<GLOBAL_AS u32u *>(gmem(p + i)) = word;
    return;
  }
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) gmem(p)[i + e] = (unsigned char)(word >> (8 * e));
}
__device__ __forceinline__ float scale_of(float peak) { return peak < 0x1p-100f ? 0.f : peak * (1.f / 448.f); }

// A wave's block of 256 elements from b on, four consecutive ones per lane; WHOLE: all of them
// exist, else lanes beyond the tensor's end hold zeros throughout and stay for the reductions.
// ODD: a second moment of the block is infinite or NaN; such a block starts again, so that the
// usual one neither keeps its inputs for it nor takes a branch between its stores (262 M elements
// 595 us so, 590 without the case, 604 to 608 with it in the one pass).
template <typename W, typename G, bool NT, bool WHOLE, bool ODD = false>
__device__ __forceinline__ void adamw8_block(const Entry<8> &t, int64_t b, float scale, const AdamWParams &p) {
  W *w = reinterpret_cast<W *>(t.w);
  const G *g = reinterpret_cast<const G *>(t.g);
  unsigned char *m = reinterpret_cast<unsigned char *>(t.m), *r = reinterpret_cast<unsigned char *>(t.v);
  const int lane = threadIdx.x & 63;
  const int64_t i = b + 4 * lane;
  const int n = WHOLE || t.n - i >= 4 ? 4 : (t.n > i ? (int)(t.n - i) : 0);
  float *ms = t.ms + b / kBlock, *vs = t.vs + b / kBlock;
  const float m_unit = *gmem(ms), r_unit = *gmem(vs);
  const f32x4 gv = load_upto4<NT>(g, i, n);
  const unsigned m_word = load_codes(m, i, n), r_word = load_codes(r, i, n);
  f32x4 wv = load_upto4<NT>(w, i, n);
  if (scale != scale) return;   // the gradient was not finite: nothing changes
  f32x4 mv = unpack_e4m3x4(m_word), rv = unpack_e4m3x4(r_word);
  {
#pragma clang fp contract(off)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = gv[e] * scale, r0 = rv[e] * r_unit;
      mv[e] = p.beta1 * (mv[e] * m_unit) + p.omb1 * x;
      rv[e] = p.beta2 * (r0 * r0) + p.omb2 * x * x;
    }
  }
  // second moments as bit patterns, in which a NaN is larger than everything
  const unsigned least = min(min(word_of(rv[0]), word_of(rv[1])), min(word_of(rv[2]), word_of(rv[3])));
  const unsigned most = max(max(word_of(rv[0]), word_of(rv[1])), max(word_of(rv[2]), word_of(rv[3])));
  if constexpr (ODD) {
    const f32x4 r0 = unpack_e4m3x4(r_word);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      rv[e] = rv[e] == __builtin_inff() ? root_of_large(r0[e] * r_unit, gv[e] * scale, p) : __builtin_sqrtf(rv[e]);
  } else if (__builtin_expect(__ballot(!(least >= word_of(0x1p-96f) && most < 0x7f800000u) && most != 0) == 0, 1)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) rv[e] = rounded_sqrt(rv[e]);
  } else {
    if (__ballot(most >= 0x7f800000u) != 0) {
      asm volatile("" ::: "memory");   // (nothing is kept: it is all loaded again)
      return adamw8_block<W, G, NT, WHOLE, true>(t, b, scale, p);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) rv[e] = __builtin_sqrtf(rv[e]);
  }
  const float decay = 1.f - p.lr * t.weight_decay;
#pragma unroll
  for (int e = 0; e < 4; ++e) wv[e] = new_weight(wv[e], mv[e], rv[e], decay, p);
  store_upto4<NT>(w, i, n, wv);
  unsigned m_nan = 0, r_nan = 0;
  if constexpr (ODD) {
    m_nan = take_out_not_finite(mv);
    r_nan = take_out_not_finite(rv);
  }
  const float m_peak = wave_peak<false>(mv), r_peak = wave_peak<true>(rv);
  float m_inv, r_inv;
  inverses(m_peak, r_peak, m_inv, r_inv);
  store_codes(m, i, n, codes_of<false>(mv, m_inv, (unsigned)i * kStepM + p.dither[0], kStepM) | m_nan);
  store_codes(r, i, n, codes_of<true>(rv, r_inv, (unsigned)i * kStepR + p.dither[1], kStepR) | r_nan);
  if (lane == 0) {
    *gmem(ms) = scale_of(m_peak);
    *gmem(vs) = scale_of(r_peak);
  }
}

template <typename W, typename G, bool NT, class TABLE>
__global__ __launch_bounds__(THREADS) void adamw8_kernel(TABLE tab, AdamWParams p) {
  const float scale = p.grad_scale ? *gmem(p.grad_scale) : 1.f;
  const int c = p.first_chunk + blockIdx.x, ti = tensor_of(tab.firsts(), tab.n, c);
  const Entry<8> t = tab.entries()[ti];   // (a copy: it comes in one round of loads, 65 gains 3.75 / 3.55 us)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t b = ((int64_t)(c - tab.firsts()[ti]) << kChunkShift) + wave * kBlock;
  if (b + kBlock <= t.n)
    adamw8_block<W, G, NT, true>(t, b, scale, p);
  else if (b < t.n)
    adamw8_block<W, G, NT, false>(t, b, scale, p);
}

// A call that moves more than this goes past the caches: nothing of it is left there when the
// next step comes, and its lines do not have to push others out.  Bytes of a call, cached
// against non-temporal (us): fp32 states 117 MB 18.7 / 21.6, 235 MB 46.1 / 41.3, 6.8 GB 1225 /
// 1135; 8-bit 114 MB 29.0 / 35.2, 236 MB 45.7 / 41.3, 3.7 GB 617 / 591.
constexpr double kCachedBytes = 128e6;

// Chunks a launch: a grid holds fewer than 2^32 threads.
constexpr int64_t kLaunchChunks = (int64_t)1 << 21;

template <int BITS, typename W, typename G, class TABLE>
hipError_t launch_typed(const TABLE &tab, int64_t chunks, bool nt, AdamWParams p, hipStream_t stream) {
  const dim3 block(THREADS);
  for (int64_t c = 0; c < chunks; c += kLaunchChunks) {
    const dim3 grid((unsigned)(chunks - c < kLaunchChunks ? chunks - c : kLaunchChunks));
    p.first_chunk = (int32_t)c;
    if constexpr (BITS == 32) {
      if (nt) hipLaunchKernelGGL((adamw32_kernel<W, G, true, TABLE>), grid, block, 0, stream, tab, p);
      else hipLaunchKernelGGL((adamw32_kernel<W, G, false, TABLE>), grid, block, 0, stream, tab, p);
    } else {
      if (nt) hipLaunchKernelGGL((adamw8_kernel<W, G, true, TABLE>), grid, block, 0, stream, tab, p);
      else hipLaunchKernelGGL((adamw8_kernel<W, G, false, TABLE>), grid, block, 0, stream, tab, p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
// How a call is launched: its types, and whether it goes past the caches.
struct Kind {
  bool weight_bf16, grad_bf16, nt;
};
template <int BITS, class TABLE>
hipError_t launch_table(const TABLE &tab, int64_t chunks, Kind k, const AdamWParams &p, hipStream_t stream) {
  if (k.weight_bf16)
    return k.grad_bf16 ? launch_typed<BITS, __bf16, __bf16>(tab, chunks, k.nt, p, stream)
                       : launch_typed<BITS, __bf16, float>(tab, chunks, k.nt, p, stream);
  return k.grad_bf16 ? launch_typed<BITS, float, __bf16>(tab, chunks, k.nt, p, stream)
                     : launch_typed<BITS, float, float>(tab, chunks, k.nt, p, stream);
}

int64_t chunks_of(int64_t n, int shift) { return (n + ((int64_t)1 << shift) - 1) >> shift; }

template <int BITS>
void fill_entry(Entry<BITS> &t, const himuon_adamw_tensor &x) {
  t.w = x.weight;
  t.g = x.grad;
  t.m = x.m;
  t.v = x.v;
  if constexpr (BITS == 8) {
    t.ms = x.m_scale;
    t.vs = x.v_scale;
  }
  t.n = x.n;
  t.weight_decay = (float)x.weight_decay;
}

template <int BITS>
void fill_table(const himuon_adamw_tensor *tensors, int32_t n_tensors, char *host) {
  int32_t *first = reinterpret_cast<int32_t *>(host);
  Entry<BITS> *t = reinterpret_cast<Entry<BITS> *>(host + entry_offset(n_tensors));
  int64_t at = 0;   // < 2^31: 2^40 elements in all and 2^24 tensors at most
  int32_t n = 0;
  for (int32_t k = 0; k < n_tensors; ++k) {
    if (tensors[k].n == 0) continue;
    first[n] = (int32_t)at;
    fill_entry<BITS>(t[n], tensors[k]);
    at += chunks_of(tensors[k].n, kChunkShift);
    ++n;
  }
  first[n] = (int32_t)at;
}

template <int BITS, int CAP>
hipError_t launch_args(const himuon_adamw_tensor *tensors, int32_t n_tensors, Kind kind, const AdamWParams &p,
                       hipStream_t stream) {
  ArgTable<BITS, CAP> tab;
  tab.n = 0;
  tab.first[0] = 0;
  auto flush = [&]() -> hipError_t {
    if (tab.n == 0) return hipSuccess;
    hipError_t e = launch_table<BITS>(tab, tab.first[tab.n], kind, p, stream);
    tab.n = 0;
    return e;
  };
  for (int32_t k = 0; k < n_tensors; ++k) {
    if (tensors[k].n == 0) continue;
    if (tab.n == CAP) {
      hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    fill_entry<BITS>(tab.t[tab.n], tensors[k]);
    tab.first[tab.n + 1] = (int32_t)(tab.first[tab.n] + chunks_of(tensors[k].n, kChunkShift));
    ++tab.n;
  }
  return flush();
}

template <int BITS>
hipError_t launch_adamw_bits(const himuon_adamw_tensor *tensors, int32_t n_tensors, bool weight_bf16, bool grad_bf16,
                             const AdamWParams &p, const void *table, hipStream_t stream) {
  int64_t total = 0;
  for (int32_t k = 0; k < n_tensors; ++k) total += tensors[k].n;
  const double each = (weight_bf16 ? 4 : 8) + (grad_bf16 ? 2 : 4) + (BITS == 8 ? 4 : 16);
  const Kind kind = {weight_bf16, grad_bf16, (double)total * each > kCachedBytes};
  if (table) {
    DeviceTable<BITS> tab{0, reinterpret_cast<const int32_t *>(table),
                          reinterpret_cast<const Entry<BITS> *>(reinterpret_cast<const char *>(table) +
                                                                entry_offset(n_tensors))};
    int64_t chunks = 0;
    for (int32_t k = 0; k < n_tensors; ++k) {
      tab.n += tensors[k].n > 0;
      chunks += chunks_of(tensors[k].n, kChunkShift);
    }
    if (chunks == 0) return hipSuccess;
    return launch_table<BITS>(tab, chunks, kind, p, stream);
  }
  return n_tensors <= kFew ? launch_args<BITS, kFew>(tensors, n_tensors, kind, p, stream)
                           : launch_args<BITS, kMost<BITS>>(tensors, n_tensors, kind, p, stream);
}

// ------------------------------------------------------------------ gradient norm
// 512 blocks of 512 threads at most, two a CU, each with four vectors a thread in flight.
// Every block ends with a release at device scope, which writes its L2 back and is paid one
// after the other: 1.07 G bf16 elements took 430 us in 2048 blocks of 256 threads and 715 us
// in 8192; 1024 blocks 377 us, these 356 us (6.0 TB/s).
constexpr int kNormThreads = 512, kNormBlocks = 512;   // each block leaves one partial sum

__device__ __forceinline__ double block_sum(double x, double *lds) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0;
  for (int k = 0; k < (int)(blockDim.x >> 6); ++k) s += lds[k];
  return s;
}

// 16 bytes of a gradient, and its squares into a sum
__device__ __forceinline__ f32x4 load_vec(const float *p) { return load4<false>(p, 0); }
__device__ __forceinline__ u16x8u load_vec(const __bf16 *p) { return *reinterpret_cast<const GLOBAL_AS u16x8u *>(gmem(p)); }
__device__ __forceinline__ void add_squares(f32x4 x, double &sum) {
#pragma unroll
  for (int e = 0; e < 4; ++e) sum = __builtin_fma((double)x[e], (double)x[e], sum);
}
__device__ __forceinline__ void add_squares(u16x8u h, double &sum) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double x = (double)bf16_bits_to_f32(h[e]);
    sum = __builtin_fma(x, x, sum);
  }
}

// Each block leaves one partial sum; the last block to finish (the ticket says which) joins
// all of them, those of the call's earlier launches among them, in a fixed order.
template <typename G>
__global__ __launch_bounds__(kNormThreads) void grad_norm_kernel(NormTable tab, double *part, int64_t before, bool last,
                                                            unsigned *ticket, double max_norm, float *out) {
  __shared__ double lds[kNormThreads / 64];
  __shared__ bool joins;
  constexpr int N = 16 / sizeof(G), STEP = N * kNormThreads;
  double sum = 0, more[3] = {0, 0, 0};
  const int chunks = tab.first[tab.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int ti = tensor_of(tab.first, tab.n, c);
    const G *g = reinterpret_cast<const G *>(tab.g[ti]);
    const int64_t base = (int64_t)(c - tab.first[ti]) << tab.shift, size = tab.size[ti];
    const int64_t end = size - base < (1 << tab.shift) ? size : base + (1 << tab.shift);
    int64_t i = base + N * threadIdx.x;
    for (; i + 3 * STEP + N <= end; i += 4 * STEP) {
      const auto a = load_vec(g + i), b = load_vec(g + i + STEP), d = load_vec(g + i + 2 * STEP), e = load_vec(g + i + 3 * STEP);
      add_squares(a, sum);
      add_squares(b, more[0]);
      add_squares(d, more[1]);
      add_squares(e, more[2]);
    }
    for (; i + N <= end; i += STEP) add_squares(load_vec(g + i), sum);
    const int64_t rest = base + (end - base) / N * N + threadIdx.x;
    if (rest < end) {
      const double x = (double)load1(g, rest);
      sum = __builtin_fma(x, x, sum);
    }
  }
  sum = block_sum(sum + more[0] + (more[1] + more[2]), lds);
  if (threadIdx.x == 0) {
    __hip_atomic_store(&part[before + blockIdx.x], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (last) {
      // (the count wraps to zero with the last block, so that the next call finds it as this one did)
      joins = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
      if (joins) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (!last) return;
  __syncthreads();
  if (!joins) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  sum = 0;
  for (int64_t i = threadIdx.x; i < before + gridDim.x; i += kNormThreads)
    sum += __hip_atomic_load(&part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = block_sum(sum, lds);
  if (threadIdx.x != 0) return;
  const double norm = __builtin_sqrt(sum);
  const bool finite = sum - sum == 0;
  gmem(out)[0] = (float)norm;
  gmem(out)[1] = finite ? (float)__builtin_fmin(1.0, max_norm / (norm + 1e-6)) : __builtin_nanf("");
}

}  // namespace

hipError_t launch_adamw(const himuon_adamw_tensor *tensors, int32_t n_tensors, bool weight_bf16, bool grad_bf16,
                        int state_bits, const AdamWParams &p, const void *table, hipStream_t stream) {
  return state_bits == 8 ? launch_adamw_bits<8>(tensors, n_tensors, weight_bf16, grad_bf16, p, table, stream)
                         : launch_adamw_bits<32>(tensors, n_tensors, weight_bf16, grad_bf16, p, table, stream);
}

size_t adamw_table_size(int32_t n_tensors, int state_bits) {
  return entry_offset(n_tensors) + (size_t)n_tensors * (state_bits == 8 ? sizeof(Entry<8>) : sizeof(Entry<32>));
}
void adamw_table(const himuon_adamw_tensor *tensors, int32_t n_tensors, int state_bits, void *host) {
  if (state_bits == 8)
    fill_table<8>(tensors, n_tensors, reinterpret_cast<char *>(host));
  else
    fill_table<32>(tensors, n_tensors, reinterpret_cast<char *>(host));
}
int adamw_few_tensors() { return kFew; }

// Chunks of the norm are long, for a block more costs its release (above): 4 M fp32 elements
// in 4 tensors take 16.1 us in chunks of 2^12, 11.8 in 2^14 and 9.9 in 2^16, 16 M bf16 ones
// 24.0, 19.9 and 14.4; 1 M in one tensor 9.9, 6.3 and 7.0.
int norm_shift_of(const himuon_grad *tensors, int32_t n_tensors) {
  int64_t total = 0;
  for (int32_t k = 0; k < n_tensors; ++k) total += tensors[k].n;
  return total <= ((int64_t)2 << 20) ? 14 : 16;
}

// The ticket, then one partial sum per block and kNormTensors tensors a launch.
size_t grad_norm_workspace(int32_t n_tensors) {
  return ((size_t)n_tensors / kNormTensors + 1) * kNormBlocks * sizeof(double) + 8;
}

hipError_t launch_grad_norm(const himuon_grad *tensors, int32_t n_tensors, bool bf16, double max_norm, float *out,
                            void *workspace, hipStream_t stream) {
  unsigned *ticket = reinterpret_cast<unsigned *>(workspace);
  double *part = reinterpret_cast<double *>(workspace) + 1;
  int64_t parts = 0;
  NormTable tab;
  tab.n = 0;
  tab.shift = norm_shift_of(tensors, n_tensors);
  tab.first[0] = 0;
  auto flush = [&](bool last) -> hipError_t {
    const int chunks = tab.first[tab.n];   // none: the last block has nothing to add of its own
    const int grid = chunks < 1 ? 1 : chunks < kNormBlocks ? chunks : kNormBlocks;
    if (bf16)
      hipLaunchKernelGGL(grad_norm_kernel<__bf16>, dim3(grid), dim3(kNormThreads), 0, stream, tab, part, parts, last, ticket,
                         max_norm, out);
    else
      hipLaunchKernelGGL(grad_norm_kernel<float>, dim3(grid), dim3(kNormThreads), 0, stream, tab, part, parts, last, ticket,
                         max_norm, out);
    parts += grid;
    tab.n = 0;
    return hipGetLastError();
  };
  for (int32_t k = 0; k < n_tensors; ++k) {
    if (tensors[k].n == 0) continue;
    if (tab.n == kNormTensors) {
      hipError_t e = flush(false);
      if (e != hipSuccess) return e;
    }
    tab.g[tab.n] = tensors[k].grad;
    tab.size[tab.n] = tensors[k].n;
    tab.first[tab.n + 1] = (int32_t)(tab.first[tab.n] + chunks_of(tensors[k].n, tab.shift));
    ++tab.n;
  }
  return flush(true);
}

}  // namespace himuon
