// AdamW over many tensors in few launches, with fp32 or 8-bit states, and the norm of many
// gradients.  Both are streams: every element of every tensor crosses HBM once.
//
// A launch covers up to kTensors tensors, whose descriptors travel in the kernel arguments
// (so a call needs no table in device memory, no upload and no wait, and pointers may
// change from step to step).  Every tensor is cut into chunks of kChunk elements, and a
// block finds the tensor of its chunk by bisection of the first-chunk table.
//
// Tensors may start at any element (views of a flattened bucket do): vectors are declared
// with the alignment of one element and the hardware takes unaligned global accesses.
#include "device_common.h"
#include "himuon_internal.h"

#include <cmath>

namespace himuon {
namespace {

using namespace dev;

constexpr int THREADS = 256;
constexpr int64_t kChunk = 4096;

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned short u16x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned u32u __attribute__((aligned(1)));

__device__ __forceinline__ float load1(const float *p, int64_t i) { return gmem(p)[i]; }
__device__ __forceinline__ float load1(const __bf16 *p, int64_t i) {
  return bf16_bits_to_f32(gmem(reinterpret_cast<const unsigned short *>(p))[i]);
}
__device__ __forceinline__ void store1(float *p, int64_t i, float x) { gmem(p)[i] = x; }
__device__ __forceinline__ void store1(__bf16 *p, int64_t i, float x) {
  gmem(reinterpret_cast<unsigned short *>(p))[i] = to_bf16_bits(x);
}
__device__ __forceinline__ f32x4 load4(const float *p, int64_t i) {
  return *reinterpret_cast<const GLOBAL_AS f32x4u *>(gmem(p + i));
}
__device__ __forceinline__ f32x4 load4(const __bf16 *p, int64_t i) {
  const u16x4u h = *reinterpret_cast<const GLOBAL_AS u16x4u *>(gmem(p + i));
  return f32x4{bf16_bits_to_f32(h[0]), bf16_bits_to_f32(h[1]), bf16_bits_to_f32(h[2]), bf16_bits_to_f32(h[3])};
}
__device__ __forceinline__ void store4(float *p, int64_t i, f32x4 x) {
  *reinterpret_cast<GLOBAL_AS f32x4u *>(gmem(p + i)) = x;
}
__device__ __forceinline__ void store4(__bf16 *p, int64_t i, f32x4 x) {
  *reinterpret_cast<GLOBAL_AS u16x4u *>(gmem(p + i)) =
      u16x4u{to_bf16_bits(x[0]), to_bf16_bits(x[1]), to_bf16_bits(x[2]), to_bf16_bits(x[3])};
}
// n (1..4) elements from i on; what lies beyond them reads as zero and is not written
template <class T>
__device__ __forceinline__ f32x4 load_upto4(const T *p, int64_t i, int n) {
  if (n >= 4) return load4(p, i);
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) x[e] = load1(p, i + e);
  return x;
}
template <class T>
__device__ __forceinline__ void store_upto4(T *p, int64_t i, int n, f32x4 x) {
  if (n >= 4) return store4(p, i, x);
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < n) store1(p, i + e, x[e]);
}

// ------------------------------------------------------------------ tables in arguments
// 8-bit entries hold two scale pointers more; both tables stay under 4 KB with the rest of
// the arguments.
template <int BITS>
struct Entry {
  void *w;
  const void *g;
  void *m, *v;
  int64_t n;
  float decay;   // 1 - lr weight_decay
};
template <>
struct Entry<8> {
  void *w;
  const void *g;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  float decay;
};
template <int BITS>
constexpr int kTensors = BITS == 8 ? 58 : 74;

template <int BITS>
struct AdamWTable {
  int32_t n;
  int32_t first[kTensors<BITS> + 1];   // first chunk of each tensor; [n]: all chunks
  Entry<BITS> t[kTensors<BITS>];
};
static_assert(sizeof(AdamWTable<32>) + sizeof(AdamWParams) <= 4096, "kernel arguments");
static_assert(sizeof(AdamWTable<8>) + sizeof(AdamWParams) <= 4096, "kernel arguments");

constexpr int kNormTensors = 200;
struct NormTable {
  int32_t n;
  int32_t first[kNormTensors + 1];
  int64_t size[kNormTensors];
  const void *g[kNormTensors];
};
static_assert(sizeof(NormTable) + 64 <= 4096, "kernel arguments");

// The tensor that chunk c belongs to: the last one whose first chunk is <= c.  (Tensors
// without elements are not in the table.)
template <class TABLE>
__device__ __forceinline__ int tensor_of(const TABLE &tab, int c) {
  int lo = 0, hi = tab.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (tab.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ AdamW
// One element: g is already scaled.  Returns the new weight; m and v are updated.
__device__ __forceinline__ float adamw(float w, float g, float &m, float &v, float &root, float decay,
                                       const AdamWParams &p) {
  m = __builtin_fmaf(p.beta1, m, p.omb1 * g);
  v = __builtin_fmaf(p.beta2, v, p.omb2 * g * g);
  root = __builtin_amdgcn_sqrtf(v);
  const float den = __builtin_fmaf(root, p.root_scale, p.eps);
  return __builtin_fmaf(w, decay, -p.step * (m * __builtin_amdgcn_rcpf(den)));
}

template <typename W, typename G>
__global__ __launch_bounds__(THREADS) void adamw32_kernel(AdamWTable<32> tab, AdamWParams p) {
  const float scale = p.grad_scale ? *gmem(p.grad_scale) : 1.f;
  if (scale != scale) return;   // the gradient was not finite: nothing changes
  const int c = blockIdx.x, ti = tensor_of(tab, c);
  const Entry<32> &t = tab.t[ti];
  W *w = reinterpret_cast<W *>(t.w);
  const G *g = reinterpret_cast<const G *>(t.g);
  float *m = reinterpret_cast<float *>(t.m), *v = reinterpret_cast<float *>(t.v);
  const int64_t base = (int64_t)(c - tab.first[ti]) * kChunk;
  const int64_t end = t.n < base + kChunk ? t.n : base + kChunk;
  for (int64_t i = base + 4 * threadIdx.x; i < end; i += 4 * THREADS) {
    const int n = end - i < 4 ? (int)(end - i) : 4;
    const f32x4 gv = load_upto4(g, i, n);
    f32x4 mv = load_upto4(m, i, n), vv = load_upto4(v, i, n), wv = load_upto4(w, i, n);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float mm = mv[e], vq = vv[e], root;
      wv[e] = adamw(wv[e], gv[e] * scale, mm, vq, root, t.decay, p);
      mv[e] = mm;
      vv[e] = vq;
    }
    store_upto4(m, i, n, mv);
    store_upto4(v, i, n, vv);
    store_upto4(w, i, n, wv);
  }
}

// ---- 8-bit states
constexpr float kE4M3Max = 448.f;
constexpr int kBlock = HIMUON_ADAMW_BLOCK;

__device__ __forceinline__ f32x4 unpack_e4m3x4(unsigned x) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, true);
  return f32x4{a[0], a[1], b[0], b[1]};
}

// Largest magnitude of a wave's values.  Magnitudes are compared as bit patterns, so that a
// NaN is larger than everything and is not lost.
__device__ __forceinline__ float wave_peak(f32x4 x) {
  unsigned k = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f = x[e];   // (a bit cast of the vector's element itself takes its first)
    k = max(k, __builtin_bit_cast(unsigned, f) & 0x7fffffffu);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) k = max(k, (unsigned)__shfl_xor((int)k, d));
  return __builtin_bit_cast(float, k);
}

// x in units of the block's scale, rounded to a neighbouring e4m3 value as the dither says:
// adding the dither below the third mantissa bit and cutting off there carries up with the
// probability of the distance to the lower neighbour.  Below 2^-6 the neighbours are 2^-9
// apart, as they are from 2^-6 to 2^-5, so such magnitudes are rounded with 2^-6 added.
__device__ __forceinline__ float dithered(float x, float inv, float least, unsigned seq) {
  const float y = __builtin_fabsf(x) * inv;
  const float low = y < 0x1p-6f ? 0x1p-6f : 0.f;
  const unsigned bits = (__builtin_bit_cast(unsigned, y + low) + ((seq >> 16) << 4 | 8u)) & ~0xfffffu;
  float q = __builtin_bit_cast(float, bits) - low;
  q = __builtin_fminf(__builtin_fmaxf(q, least), kE4M3Max);
  return x != 0.f && inv > 0.f ? __builtin_copysignf(q, x) : 0.f;
}

// One wave's block of 256 elements: four consecutive ones per lane.
template <class T>
__device__ __forceinline__ unsigned hold(f32x4 x, int n, float least, unsigned seq, unsigned mult, T *code,
                                         int64_t i, float *scale) {
  float peak = wave_peak(x);
  if (peak < 0x1p-100f) peak = 0.f;
  const float inv = peak > 0.f ? kE4M3Max / peak : (peak == 0.f ? 0.f : peak);   // NaN stays NaN
  f32x4 q;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = dithered(x[e], inv, least, seq + e * mult);
  const unsigned word = pack_fp8x4(q[0], q[1], q[2], q[3], 1.f);
  if (n >= 4) {
    *reinterpret_cast<GLOBAL_AS u32u *>(gmem(code + i)) = word;
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) gmem(code)[i + e] = (unsigned char)(word >> (8 * e));
  }
  if ((threadIdx.x & 63) == 0) *gmem(scale) = peak * (1.f / kE4M3Max);
  return word;
}

__device__ __forceinline__ f32x4 load_codes(const unsigned char *p, int64_t i, int n) {
  unsigned word = 0;
  if (n >= 4) {
    word = *reinterpret_cast<const GLOBAL_AS u32u *>(gmem(p + i));
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < n) word |= (unsigned)gmem(p)[i + e] << (8 * e);
  }
  return unpack_e4m3x4(word);
}

template <typename W, typename G>
__global__ __launch_bounds__(THREADS) void adamw8_kernel(AdamWTable<8> tab, AdamWParams p) {
  const float scale = p.grad_scale ? *gmem(p.grad_scale) : 1.f;
  if (scale != scale) return;   // the gradient was not finite: nothing changes
  const int c = blockIdx.x, ti = tensor_of(tab, c);
  const Entry<8> &t = tab.t[ti];
  W *w = reinterpret_cast<W *>(t.w);
  const G *g = reinterpret_cast<const G *>(t.g);
  unsigned char *m = reinterpret_cast<unsigned char *>(t.m), *r = reinterpret_cast<unsigned char *>(t.v);
  const int64_t base = (int64_t)(c - tab.first[ti]) * kChunk;
  const int64_t end = t.n < base + kChunk ? t.n : base + kChunk;
  const int lane = threadIdx.x & 63;
  // a wave takes whole blocks: every lane stays in the loop until its wave's block is done
  for (int64_t b = base + (int64_t)(threadIdx.x >> 6) * kBlock; b < end; b += THREADS / 64 * kBlock) {
    const int64_t i = b + 4 * lane;
    const int n = end - i >= 4 ? 4 : (end > i ? (int)(end - i) : 0);
    float *ms = t.ms + b / kBlock, *vs = t.vs + b / kBlock;
    const float m_unit = *gmem(ms), r_unit = *gmem(vs);
    const f32x4 gv = load_upto4(g, i, n);
    f32x4 mv = load_codes(m, i, n), rv = load_codes(r, i, n), wv = load_upto4(w, i, n);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float r0 = rv[e] * r_unit;
      float mm = mv[e] * m_unit, vq = r0 * r0, root;
      wv[e] = adamw(wv[e], gv[e] * scale, mm, vq, root, t.decay, p);
      // lanes beyond the tensor's end hold zeros throughout
      mv[e] = mm;
      rv[e] = root;
    }
    const unsigned at = (unsigned)i;   // the sequences are taken modulo 2^32
    hold(mv, n, 0.f, at * 0x9E3779B1u + p.dither[0], 0x9E3779B1u, m, i, ms);
    hold(rv, n, 0x1p-9f, at * 0x85EBCA6Bu + p.dither[1], 0x85EBCA6Bu, r, i, vs);
    store_upto4(w, i, n, wv);
  }
}

template <int BITS, typename W, typename G>
void launch_table(const AdamWTable<BITS> &tab, const AdamWParams &p, hipStream_t stream) {
  const dim3 grid((unsigned)tab.first[tab.n]);
  if constexpr (BITS == 32)
    hipLaunchKernelGGL((adamw32_kernel<W, G>), grid, dim3(THREADS), 0, stream, tab, p);
  else
    hipLaunchKernelGGL((adamw8_kernel<W, G>), grid, dim3(THREADS), 0, stream, tab, p);
}

template <int BITS>
hipError_t launch_adamw_bits(const himuon_adamw_tensor *tensors, int32_t n_tensors, bool weight_bf16, bool grad_bf16,
                             double lr, const AdamWParams &p, hipStream_t stream) {
  AdamWTable<BITS> tab;
  tab.n = 0;
  tab.first[0] = 0;
  auto flush = [&]() -> hipError_t {
    if (tab.n == 0) return hipSuccess;
    if (weight_bf16)
      grad_bf16 ? launch_table<BITS, __bf16, __bf16>(tab, p, stream) : launch_table<BITS, __bf16, float>(tab, p, stream);
    else
      grad_bf16 ? launch_table<BITS, float, __bf16>(tab, p, stream) : launch_table<BITS, float, float>(tab, p, stream);
    tab.n = 0;
    return hipGetLastError();
  };
  for (int32_t k = 0; k < n_tensors; ++k) {
    const himuon_adamw_tensor &x = tensors[k];
    if (x.n == 0) continue;
    const int64_t chunks = (x.n + kChunk - 1) / kChunk;   // of all tensors: < 2^29 (n is 2^40 in all at most)
    if (tab.n == kTensors<BITS>) {
      hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    Entry<BITS> &t = tab.t[tab.n];
    t.w = x.weight;
    t.g = x.grad;
    t.m = x.m;
    t.v = x.v;
    if constexpr (BITS == 8) {
      t.ms = x.m_scale;
      t.vs = x.v_scale;
    }
    t.n = x.n;
    t.decay = (float)(1.0 - lr * x.weight_decay);
    tab.first[tab.n + 1] = (int32_t)(tab.first[tab.n] + chunks);
    ++tab.n;
  }
  return flush();
}

// ------------------------------------------------------------------ gradient norm
constexpr int kNormBlocks = 2048;   // blocks of a launch at most; each leaves one partial sum

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}
__device__ __forceinline__ double block_sum(double x, double *lds) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0;
  for (int k = 0; k < (int)(blockDim.x >> 6); ++k) s += lds[k];
  return s;
}

template <typename G>
__global__ __launch_bounds__(THREADS) void grad_norm_kernel(NormTable tab, double *part) {
  __shared__ double lds[THREADS / 64];
  double sum = 0;
  const int chunks = tab.first[tab.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int ti = tensor_of(tab, c);
    const G *g = reinterpret_cast<const G *>(tab.g[ti]);
    const int64_t base = (int64_t)(c - tab.first[ti]) * kChunk, size = tab.size[ti];
    const int64_t end = size < base + kChunk ? size : base + kChunk;
    for (int64_t i = base + 4 * threadIdx.x; i < end; i += 4 * THREADS) {
      const f32x4 x = load_upto4(g, i, end - i < 4 ? (int)(end - i) : 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = __builtin_fma((double)x[e], (double)x[e], sum);
    }
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) gmem(part)[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void grad_norm_join_kernel(const double *part, int64_t n, double max_norm,
                                                              float *out) {
  __shared__ double lds[16];
  double sum = 0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) sum += gmem(part)[i];
  sum = block_sum(sum, lds);
  if (threadIdx.x != 0) return;
  const double norm = __builtin_sqrt(sum);
  const bool finite = sum - sum == 0;
  gmem(out)[0] = (float)norm;
  gmem(out)[1] = finite ? (float)__builtin_fmin(1.0, max_norm / (norm + 1e-6)) : __builtin_nanf("");
}

}  // namespace

hipError_t launch_adamw(const himuon_adamw_tensor *tensors, int32_t n_tensors, bool weight_bf16, bool grad_bf16,
                        int state_bits, double lr, const AdamWParams &p, hipStream_t stream) {
  return state_bits == 8 ? launch_adamw_bits<8>(tensors, n_tensors, weight_bf16, grad_bf16, lr, p, stream)
                         : launch_adamw_bits<32>(tensors, n_tensors, weight_bf16, grad_bf16, lr, p, stream);
}

// One partial sum per block, kNormTensors tensors a launch.
size_t grad_norm_workspace(int32_t n_tensors) {
  return ((size_t)n_tensors / kNormTensors + 1) * kNormBlocks * sizeof(double);
}

hipError_t launch_grad_norm(const himuon_grad *tensors, int32_t n_tensors, bool bf16, double max_norm, float *out,
                            void *workspace, hipStream_t stream) {
  double *part = reinterpret_cast<double *>(workspace);
  int64_t parts = 0;
  NormTable tab;
  tab.n = 0;
  tab.first[0] = 0;
  auto flush = [&]() -> hipError_t {
    if (tab.n == 0) return hipSuccess;
    const int grid = tab.first[tab.n] < kNormBlocks ? tab.first[tab.n] : kNormBlocks;
    if (bf16)
      hipLaunchKernelGGL(grad_norm_kernel<__bf16>, dim3(grid), dim3(THREADS), 0, stream, tab, part + parts);
    else
      hipLaunchKernelGGL(grad_norm_kernel<float>, dim3(grid), dim3(THREADS), 0, stream, tab, part + parts);
    parts += grid;
    tab.n = 0;
    return hipGetLastError();
  };
  for (int32_t k = 0; k < n_tensors; ++k) {
    if (tensors[k].n == 0) continue;
    const int64_t chunks = (tensors[k].n + kChunk - 1) / kChunk;
    if (tab.n == kNormTensors) {
      hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    tab.g[tab.n] = tensors[k].grad;
    tab.size[tab.n] = tensors[k].n;
    tab.first[tab.n + 1] = (int32_t)(tab.first[tab.n] + chunks);
    ++tab.n;
  }
  hipError_t e = flush();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_norm_join_kernel, dim3(1), dim3(1024), 0, stream, part, parts, max_norm, out);
  return hipGetLastError();
}

}  // namespace himuon
