// clip.hip -- global norm and clipping of many gradient tensors
// (include/ssm_train.h).
//
// Two passes over the data, both bound by memory: the sum of squares (one
// partial sum per workgroup, in 64 bits, so that neither the length of the
// sum nor the size of the gradients costs digits), then the scaling, each of
// whose workgroups first adds the partial sums in the same fixed order.  The
// scaling walks the tensors from the end, so that what the first pass read
// last, and the caches still hold, is read first.  51.5 million fp32 elements in
// 60 tensors: 103 us, of it 40 the sum (0.21 GB at 5.1 TB/s).
//
// Few elements (kSmall, in a few tensors) are one workgroup's work: it adds
// and then scales in one launch (fp32, 4 tensors: 16000 elements 5.1 us against
// 8.4 us for two launches, 64000 9.7 against 11.6, 128000 14.7 against 11.1).
//
// The tensor table travels in the kernel arguments, kTable tensors a launch:
// nothing is copied to the device, and a captured launch keeps its own.
#include <math.h>
#include <stdint.h>

#include "../../include/ssm_train.h"
#include "abi_util.hpp"
#include "ssm_common.hpp"

namespace ssm {

namespace {

constexpr int kTable = 96;             // tensors a launch (3 KB of arguments)
constexpr int kBlock = 8192;           // elements a workgroup takes at a time
constexpr int64_t kSmall = 65536;      // elements of the one-launch form,
constexpr int kSmallCount = 16;        // which walks its tensors one by one
constexpr int64_t kMaxWgs = 1024;      // per launch: also its partial sums
constexpr int32_t kMaxTensors = 65536;
constexpr int64_t kMaxElems = int64_t(1) << 40;

struct Table {
  int count;
  int64_t blocks;         // of all its tensors
  const void* in[kTable];
  void* out[kTable];
  int64_t n[kTable];
  int64_t first[kTable];  // first block of each tensor
};

struct Piece {
  int tensor;
  int64_t e0;  // first element
  int n;       // elements
};

// The tensor of block b: the last one whose first block is at most b (empty
// tensors share the next one's first block and come before it).
__device__ __forceinline__ Piece piece_of(const Table& t, int64_t b) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= b) lo = mid;
    else hi = mid - 1;
  }
  const int64_t e0 = (b - t.first[lo]) * kBlock;
  const int64_t left = t.n[lo] - e0;
  return Piece{lo, e0, static_cast<int>(left < kBlock ? left : kBlock)};
}

template <class T> struct Vec;  // 16 bytes
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float* f) {
    return uint4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};
template <> struct Vec<bf16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
      w[i] = f32_to_bf16(f[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(f[2 * i + 1])) << 16);
    return uint4{w[0], w[1], w[2], w[3]};
  }
};

typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4;
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint4* p) {
  const u32x4* const q = reinterpret_cast<const u32x4*>(p);
  return __builtin_bit_cast(uint4, STREAM ? __builtin_nontemporal_load(q) : *q);
}
template <bool STREAM>
__device__ __forceinline__ void store16(uint4* p, uint4 v) {
  u32x4* const q = reinterpret_cast<u32x4*>(p);
  if (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), q);
  else *q = __builtin_bit_cast(u32x4, v);
}

__device__ __forceinline__ double wg_sum(double s, double* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = s;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

template <class T>
__global__ __launch_bounds__(256) void k_square_sums(Table t, double* __restrict__ part) {
  __shared__ double red[4];
  constexpr int N = Vec<T>::N, U = kBlock / (256 * N);
  double s = 0.0;
  for (int64_t b = blockIdx.x; b < t.blocks; b += gridDim.x) {
    const Piece p = piece_of(t, b);
    const T* const src = static_cast<const T*>(t.in[p.tensor]) + p.e0;
    if (p.n == kBlock) {
      uint4 u[U];
#pragma unroll
      for (int i = 0; i < U; i++) u[i] = reinterpret_cast<const uint4*>(src)[threadIdx.x + 256 * i];
#pragma unroll
      for (int i = 0; i < U; i++) {
        float f[N];
        Vec<T>::get(u[i], f);
#pragma unroll
        for (int e = 0; e < N; e++) s = fma(static_cast<double>(f[e]), static_cast<double>(f[e]), s);
      }
    } else {
      for (int e = threadIdx.x; e < p.n; e += 256) {
        const double v = load_io(src + e);
        s = fma(v, v, s);
      }
    }
  }
  s = wg_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The factor of the scaling; 1 where nothing is clipped.
__device__ __forceinline__ float clip_factor(double total, float max_norm) {
  const bool clip = total > static_cast<double>(max_norm) && isfinite(total);
  return clip ? static_cast<float>(static_cast<double>(max_norm) / total) : 1.0f;
}

// Both passes over a table of at most kSmall elements, one workgroup.
template <class T>
__global__ __launch_bounds__(1024) void k_clip_small(Table t, float max_norm, int scale, float* __restrict__ norm) {
  __shared__ double red[16];
  constexpr int N = Vec<T>::N;
  double s = 0.0;
  for (int i = 0; i < t.count; i++) {
    const T* const src = static_cast<const T*>(t.in[i]);
    const int n = static_cast<int>(t.n[i]), nv = n / N;
#pragma unroll 2
    for (int e = threadIdx.x; e < nv; e += 1024) {
      float f[N];
      Vec<T>::get(reinterpret_cast<const uint4*>(src)[e], f);
#pragma unroll
      for (int k = 0; k < N; k++) s = fma(static_cast<double>(f[k]), static_cast<double>(f[k]), s);
    }
    if (static_cast<int>(threadIdx.x) < n - nv * N) {
      const double v = load_io(src + nv * N + threadIdx.x);
      s = fma(v, v, s);
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < 16; w++) s += red[w];
  const double total = sqrt(s);
  if (threadIdx.x == 0) *norm = static_cast<float>(total);
  if (!scale) return;
  const float c = clip_factor(total, max_norm);
  for (int i = 0; i < t.count; i++) {
    const T* const src = static_cast<const T*>(t.in[i]);
    T* const dst = static_cast<T*>(t.out[i]);
    if (c == 1.0f && dst == src) continue;
    const int n = static_cast<int>(t.n[i]), nv = n / N;
#pragma unroll 2
    for (int e = threadIdx.x; e < nv; e += 1024) {
      float f[N];
      Vec<T>::get(reinterpret_cast<const uint4*>(src)[e], f);
#pragma unroll
      for (int k = 0; k < N; k++) f[k] = c == 1.0f ? f[k] : f[k] * c;
      reinterpret_cast<uint4*>(dst)[e] = Vec<T>::put(f);
    }
    if (static_cast<int>(threadIdx.x) < n - nv * N) {
      const float f = load_io(src + nv * N + threadIdx.x);
      store_io(dst + nv * N + threadIdx.x, c == 1.0f ? f : f * c);
    }
  }
}

// STREAM: past the caches, so that the outputs leave them to the inputs that
// the sum has just read.
template <class T, bool STREAM>
__global__ __launch_bounds__(256) void k_clip_scale(Table t, const double* __restrict__ part, int nparts,
                                                   float max_norm, int scale, float* __restrict__ norm) {
  __shared__ double red[4];
  constexpr int N = Vec<T>::N, U = kBlock / (256 * N);
  double s = 0.0;
  for (int i = threadIdx.x; i < nparts; i += 256) s += part[i];
  const double total = sqrt(wg_sum(s, red));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  if (!scale) return;
  const float c = clip_factor(total, max_norm);
  const bool clip = c != 1.0f;
  for (int64_t i = blockIdx.x; i < t.blocks; i += gridDim.x) {
    const Piece p = piece_of(t, t.blocks - 1 - i);
    const T* const src = static_cast<const T*>(t.in[p.tensor]) + p.e0;
    T* const dst = static_cast<T*>(t.out[p.tensor]) + p.e0;
    if (!clip && dst == src) continue;
    if (p.n == kBlock) {
      uint4 u[U];
#pragma unroll
      for (int j = 0; j < U; j++) u[j] = load16<STREAM>(reinterpret_cast<const uint4*>(src) + threadIdx.x + 256 * j);
#pragma unroll
      for (int j = 0; j < U; j++) {
        float f[N];
        Vec<T>::get(u[j], f);
#pragma unroll
        for (int e = 0; e < N; e++) f[e] = clip ? f[e] * c : f[e];
        store16<STREAM>(reinterpret_cast<uint4*>(dst) + threadIdx.x + 256 * j, Vec<T>::put(f));
      }
    } else {
      for (int e = threadIdx.x; e < p.n; e += 256) {
        const float f = load_io(src + e);
        store_io(dst + e, clip ? f * c : f);
      }
    }
  }
}

int64_t launches_for(int32_t count) { return (count + kTable - 1) / kTable; }

unsigned wgs_for(const Table& t) {
  return static_cast<unsigned>(t.blocks < 1 ? 1 : t.blocks < kMaxWgs ? t.blocks : kMaxWgs);
}

bool check_counts(int32_t count, const int64_t* n) {
  if (count < 1 || count > kMaxTensors || !n) return false;
  for (int32_t i = 0; i < count; i++)
    if (n[i] < 0 || n[i] > kMaxElems) return false;
  return true;
}

Table table_of(int32_t first, int32_t count, const void* const* in, void* const* out, const int64_t* n) {
  Table t{};
  const int32_t left = count - first;
  t.count = left < kTable ? left : kTable;
  for (int i = 0; i < t.count; i++) {
    t.in[i] = in[first + i];
    t.out[i] = out ? out[first + i] : nullptr;
    t.n[i] = n[first + i];
    t.first[i] = t.blocks;
    t.blocks += (n[first + i] + kBlock - 1) / kBlock;
  }
  return t;
}

template <class T>
hipError_t run_clip(int32_t count, const void* const* in, void* const* out, const int64_t* n, float max_norm,
                    float* norm, double* part, hipStream_t st) {
  int64_t total = 0;
  for (int32_t i = 0; i < count; i++) total += n[i];
  if (count <= kSmallCount && total <= kSmall) {
    k_clip_small<T><<<1, 1024, 0, st>>>(table_of(0, count, in, out, n), max_norm, out ? 1 : 0, norm);
    return hipGetLastError();
  }
  int nparts = 0;
  for (int32_t i = 0; i < count; i += kTable) {
    const Table t = table_of(i, count, in, out, n);
    const unsigned g = wgs_for(t);
    k_square_sums<T><<<g, 256, 0, st>>>(t, part + nparts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    nparts += static_cast<int>(g);
  }
  // Gradients of three quarters of the 256 MB cache or more leave no room for
  // what reads the outputs next.  fp32, cached and streamed, alone and with a
  // pass over the outputs behind: 96 MB 61 and 53, 106 and 110 us; 160 MB 100 and
  // 82, 161 and 171; 208 MB 128 and 105, 214 and 215; 320 MB 194 and 157, 322 and 313.
  const bool stream = total * static_cast<int64_t>(sizeof(T)) >= (int64_t(192) << 20);
  const int32_t last = static_cast<int32_t>((launches_for(count) - 1) * kTable);
  for (int32_t i = last; i >= 0; i -= kTable) {
    const Table t = table_of(i, count, in, out, n);
    const auto k = stream ? k_clip_scale<T, true> : k_clip_scale<T, false>;
    k<<<out ? wgs_for(t) : 1u, 256, 0, st>>>(t, part, nparts, max_norm, out ? 1 : 0, i == last ? norm : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !out) return e;
  }
  return hipSuccess;
}

}  // namespace

}  // namespace ssm

extern "C" {

size_t ssm_clip_grads_workspace_bytes(int32_t count, const int64_t* n) {
  if (!ssm::check_counts(count, n)) return 0;
  return abi::align_up(static_cast<size_t>(ssm::launches_for(count) * ssm::kMaxWgs) * sizeof(double));
}

ssm_status ssm_clip_grads(int32_t count, const void* const* in, void* const* out, const int64_t* n, int32_t io,
                          float max_norm, float* norm, void* ws, size_t ws_bytes, void* stream) {
  if (!ssm::check_counts(count, n) || !in || !abi::good(norm) || !(max_norm > 0.0f)) return SSM_ERR_ARG;
  if (io != SSM_F32 && io != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < count; i++) {
    if (n[i] == 0) continue;
    if (!abi::good(in[i]) || (out && !abi::good(out[i]))) return SSM_ERR_ARG;
  }
  const ssm_status s = abi::check_ws(ws, ws_bytes, ssm_clip_grads_workspace_bytes(count, n));
  if (s != SSM_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(ws);
  const hipError_t e = io == SSM_BF16 ? ssm::run_clip<ssm::bf16_t>(count, in, out, n, max_norm, norm, part, st)
                                      : ssm::run_clip<float>(count, in, out, n, max_norm, norm, part, st);
  return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
