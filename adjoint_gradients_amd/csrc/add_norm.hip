// add_norm.hip -- the residual update with the RMS norm of the next layer's
// input, and its gradient (include/ssm_train.h).
//
// Both are bound by HBM: each element is read and written once.  A row is
// held in the registers of TPR lanes, NE elements a lane, between its sum of
// squares and its scaling, so nothing is read twice.  A workgroup walks rows
// with the scale (and, in the gradient, its column sums of d norm_scale) in
// registers.  With u = norm_scale dx and xh = r rinv:
//   dr = dr_out + rinv (u - xh mean(u xh)),  dnorm_scale = sum_t dx xh.
// All sums are fp32 (column sums over a workgroup's rows, then 64 bits).
// 65536 rows, bf16: 292 us at 2048 channels (1.6 GB, 5.5 TB/s), gradient 251 us
// at 1536 (1.4 GB, 5.6 TB/s); 5 rows of 2048: 3.6 us, a launch.
#include <math.h>
#include <stdint.h>

#include "../../include/ssm_train.h"
#include "abi_util.hpp"
#include "ssm_common.hpp"

namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 4;  // elements an access
constexpr int64_t kMaxP = 16384;
constexpr int64_t kMaxRows = int64_t(1) << 31;

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;

typedef __attribute__((__vector_size__(4 * sizeof(float)), aligned(4))) float f32x4_any;
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)), aligned(2))) uint32_t u32x2_any;
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;

// The next four of a row's `left` > 0 elements as floats, zeros past its end.
// AL: rows start aligned and hold a multiple of four; otherwise the accesses
// are aligned to the element only, and a row's last ones are single.
template <bool AL>
__device__ __forceinline__ void load_vec(const float* p, int left, float* o) {
  if (AL || left >= 4) {
    const f32x4 v = AL ? *reinterpret_cast<const f32x4*>(p) : f32x4(*reinterpret_cast<const f32x4_any*>(p));
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = v[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = e < left ? p[e] : 0.0f;
  }
}
template <bool AL>
__device__ __forceinline__ void load_vec(const bf16_t* p, int left, float* o) {
  if (AL || left >= 4) {
    const u32x2 u = AL ? *reinterpret_cast<const u32x2*>(p) : u32x2(*reinterpret_cast<const u32x2_any*>(p));
    o[0] = __uint_as_float(u[0] << 16); o[1] = __uint_as_float(u[0] & 0xffff0000u);
    o[2] = __uint_as_float(u[1] << 16); o[3] = __uint_as_float(u[1] & 0xffff0000u);
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = e < left ? bf16_to_f32(p[e]) : 0.0f;
  }
}
template <bool AL>
__device__ __forceinline__ void store_vec(float* p, int left, const float* v) {
  if (AL) {
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  } else if (left >= 4) {
    *reinterpret_cast<f32x4_any*>(p) = f32x4_any{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (e < left) p[e] = v[e];
  }
}
template <bool AL>
__device__ __forceinline__ void store_vec(bf16_t* p, int left, const float* v) {
  const uint32_t a = f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16);
  const uint32_t b = f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
  if (AL) {
    *reinterpret_cast<u32x2*>(p) = u32x2{a, b};
  } else if (left >= 4) {
    *reinterpret_cast<u32x2_any*>(p) = u32x2_any{a, b};
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (e < left) p[e] = static_cast<bf16_t>((e < 2 ? a : b) >> (e % 2 * 16));
  }
}

// Sum over the TPR lanes of a row; every one of them gets it.  buf: one float
// per wavefront, used alternately by successive calls.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  if constexpr (TPR > 64) {
    if (threadIdx.x % 64 == 0) buf[threadIdx.x / 64] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; w++) v += buf[w];
  }
  return v;
}

template <class T, int TPR, int NE, bool AL>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void k_add_norm(
    int64_t rows, int P, const float* r, const T* __restrict__ y, const float* __restrict__ scale, float eps,
    float* r_out, T* __restrict__ x, float* __restrict__ rinv) {
  constexpr int NT = TPR > kThreads ? TPR : kThreads;
  constexpr int RW = NT / TPR;  // rows a workgroup holds at once
  constexpr int NV = NE / kVec;
  __shared__ float buf[2][NT / 64];
  const int l = threadIdx.x % TPR;
  float gm[NE];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int p = (l + TPR * i) * kVec;
    if (p < P) load_vec<AL>(scale + p, P - p, gm + i * kVec);
  }
  const float inv_p = 1.0f / static_cast<float>(P);
  int flip = 0;
  // whole wavefronts leave together; with TPR > 64 the workgroup has one row
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * RW + threadIdx.x / TPR; t < rows;
       t += static_cast<int64_t>(gridDim.x) * RW, flip ^= 1) {
    const int64_t o = t * P;
    float v[NE], u[NE];
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int p = (l + TPR * i) * kVec;
      if (p < P) load_vec<AL>(r + o + p, P - p, v + i * kVec);
    }
    if (y) {
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const int p = (l + TPR * i) * kVec;
        if (p < P) load_vec<AL>(y + o + p, P - p, u + i * kVec);
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int p = (l + TPR * i) * kVec;
      if (p < P) {
#pragma unroll
        for (int e = 0; e < kVec; e++) {
          if (y) v[i * kVec + e] += u[i * kVec + e];
          ss = fmaf(v[i * kVec + e], v[i * kVec + e], ss);
        }
        if (r_out) store_vec<AL>(r_out + o + p, P - p, v + i * kVec);
      }
    }
    ss = row_sum<TPR>(ss, buf[flip]);
    const float ri = 1.0f / sqrtf(fmaf(ss, inv_p, eps));
    if (rinv && l == 0) rinv[t] = ri;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int p = (l + TPR * i) * kVec;
      if (p < P) {
#pragma unroll
        for (int e = 0; e < kVec; e++) v[i * kVec + e] = gm[i * kVec + e] * (v[i * kVec + e] * ri);
        store_vec<AL>(x + o + p, P - p, v + i * kVec);
      }
    }
  }
}

template <class T, int TPR, int NE, bool AL>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void k_add_norm_grad(
    int64_t rows, int P, const float* __restrict__ r, const float* __restrict__ rinv, const float* __restrict__ scale,
    const T* __restrict__ dx, const float* dr_out, float* dr, float* __restrict__ part) {
  constexpr int NT = TPR > kThreads ? TPR : kThreads;
  constexpr int RW = NT / TPR;
  constexpr int NV = NE / kVec;
  __shared__ float buf[2][NT / 64];
  __shared__ float cols[RW > 1 ? TPR * NE : 1];
  const int l = threadIdx.x % TPR;
  float gm[NE], dg[NE];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int p = (l + TPR * i) * kVec;
    if (p < P) load_vec<AL>(scale + p, P - p, gm + i * kVec);
  }
#pragma unroll
  for (int e = 0; e < NE; e++) dg[e] = 0.0f;
  const float inv_p = 1.0f / static_cast<float>(P);
  int flip = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * RW + threadIdx.x / TPR; t < rows;
       t += static_cast<int64_t>(gridDim.x) * RW, flip ^= 1) {
    const int64_t o = t * P;
    float xh[NE], d[NE], c[NE];
    const float ri = rinv[t];
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int p = (l + TPR * i) * kVec;
      if (p < P) {
        load_vec<AL>(r + o + p, P - p, xh + i * kVec);
        load_vec<AL>(dx + o + p, P - p, d + i * kVec);
        if (dr_out) load_vec<AL>(dr_out + o + p, P - p, c + i * kVec);
      }
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      if ((l + TPR * i) * kVec < P) {
#pragma unroll
        for (int e = 0; e < kVec; e++) {
          const int k = i * kVec + e;
          xh[k] *= ri;
          dg[k] = fmaf(d[k], xh[k], dg[k]);
          d[k] *= gm[k];
          m = fmaf(d[k], xh[k], m);
        }
      }
    }
    m = row_sum<TPR>(m, buf[flip]) * inv_p;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int p = (l + TPR * i) * kVec;
      if (p < P) {
#pragma unroll
        for (int e = 0; e < kVec; e++) {
          const int k = i * kVec + e;
          const float g = ri * fmaf(-xh[k], m, d[k]);
          d[k] = dr_out ? c[k] + g : g;
        }
        store_vec<AL>(dr + o + p, P - p, d + i * kVec);
      }
    }
  }
  if (!part) return;
  // the workgroup's column sums: its row groups one after another
  if constexpr (RW > 1) {
    for (int w = 0; w < RW; w++) {
      if (static_cast<int>(threadIdx.x) / TPR == w) {
#pragma unroll
        for (int e = 0; e < NE; e++) {
          const int k = e * TPR + l;
          cols[k] = w == 0 ? dg[e] : cols[k] + dg[e];
        }
      }
      __syncthreads();
    }
    if (threadIdx.x < TPR) {
#pragma unroll
      for (int e = 0; e < NE; e++) dg[e] = cols[e * TPR + l];
    }
  }
  if (threadIdx.x < TPR) {
    float* const q = part + static_cast<int64_t>(blockIdx.x) * P;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
      for (int e = 0; e < kVec; e++) {
        const int p = (l + TPR * i) * kVec + e;
        if (p < P) q[p] = dg[i * kVec + e];
      }
  }
}

// out[p] = sum over nb rows of part, in 64 bits: 16 columns by 16 row groups a workgroup.
__global__ __launch_bounds__(256) void k_column_sums(int nb, int P, const float* __restrict__ part,
                                                    float* __restrict__ out) {
  __shared__ double red[16][17];
  const int c = threadIdx.x % 16, g = threadIdx.x / 16;
  const int p = static_cast<int>(blockIdx.x) * 16 + c;
  double s = 0.0;
  if (p < P) {
#pragma unroll 8
    for (int b = g; b < nb; b += 16) s += part[static_cast<int64_t>(b) * P + p];
  }
  red[g][c] = s;
  __syncthreads();
  if (g == 0 && p < P) {
    for (int i = 1; i < 16; i++) s += red[i][c];
    out[p] = static_cast<float>(s);
  }
}

// Lanes a row and elements a lane: eight elements (sixteen for the widest
// rows) and as many lanes as the row needs, in steps; more elements a lane
// leave fewer wavefronts in flight (65536 rows of 2048: 298 us with 256 lanes
// of 8, 352 with 64 of 32).  Narrow rows go four to a workgroup if there are
// many (65536 rows of 512: 77 us with 64 lanes a row, 83 with 256; 64 rows:
// 3.2 and 2.9).
struct Shape {
  int tpr, ne, rows_wg;
};

Shape shape_for(int64_t T, int64_t P) {
  if (P <= 512 && T >= 1024) return Shape{64, 8, 4};
  if (P <= 2048) return Shape{256, 8, 1};
  if (P <= 4096) return Shape{512, 8, 1};
  if (P <= 8192) return Shape{1024, 8, 1};
  return Shape{1024, 16, 1};
}

constexpr int64_t kFwdWgs = 4096, kGradWgs = 1024;

unsigned grid_for(const Shape& s, int64_t T, int64_t most) {
  const int64_t w = (T + s.rows_wg - 1) / s.rows_wg;
  return static_cast<unsigned>(w < most ? w : most);
}

struct NormArgs {
  int64_t T, P;
  const float* r;
  const void* y;      // forward: y; gradient: dx
  const float* scale;
  float eps;
  float* r_out;       // gradient: dr
  void* x;
  float* rinv;
  const float* rinv_in;
  const float* dr_out;
  float* part;
};

template <bool GRAD, class T, int TPR, int NE, bool AL>
hipError_t launch_shape(const NormArgs& a, unsigned grid, hipStream_t st) {
  constexpr int NT = TPR > kThreads ? TPR : kThreads;
  if constexpr (GRAD)
    k_add_norm_grad<T, TPR, NE, AL><<<grid, NT, 0, st>>>(a.T, static_cast<int>(a.P), a.r, a.rinv_in, a.scale,
                                                        static_cast<const T*>(a.y), a.dr_out, a.r_out, a.part);
  else
    k_add_norm<T, TPR, NE, AL><<<grid, NT, 0, st>>>(a.T, static_cast<int>(a.P), a.r, static_cast<const T*>(a.y),
                                                   a.scale, a.eps, a.r_out, static_cast<T*>(a.x), a.rinv);
  return hipGetLastError();
}

template <bool GRAD, class T, bool AL>
hipError_t launch_vec(const NormArgs& a, const Shape& s, unsigned grid, hipStream_t st) {
  if (s.tpr == 64) return launch_shape<GRAD, T, 64, 8, AL>(a, grid, st);
  if (s.tpr == 256) return launch_shape<GRAD, T, 256, 8, AL>(a, grid, st);
  if (s.tpr == 512) return launch_shape<GRAD, T, 512, 8, AL>(a, grid, st);
  if (s.ne == 8) return launch_shape<GRAD, T, 1024, 8, AL>(a, grid, st);
  return launch_shape<GRAD, T, 1024, 16, AL>(a, grid, st);
}

// Rows of P elements start 16 bytes aligned in float32, 8 in bfloat16, when P
// is a multiple of 4.  (65536 rows of 999: 181 us; 305 with one element an access.)
template <bool GRAD>
hipError_t launch_norm(const NormArgs& a, bool bf16, hipStream_t st) {
  const Shape s = shape_for(a.T, a.P);
  const unsigned grid = grid_for(s, a.T, GRAD ? kGradWgs : kFwdWgs);
  if (a.P % 4 == 0)
    return bf16 ? launch_vec<GRAD, bf16_t, true>(a, s, grid, st) : launch_vec<GRAD, float, true>(a, s, grid, st);
  return bf16 ? launch_vec<GRAD, bf16_t, false>(a, s, grid, st) : launch_vec<GRAD, float, false>(a, s, grid, st);
}

ssm_status check_sizes(int64_t T, int64_t P) {
  if (T < 1 || P < 1) return SSM_ERR_ARG;
  if (P > kMaxP || T > kMaxRows) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

size_t grad_bytes(int64_t T, int64_t P) {
  return abi::align_up(static_cast<size_t>(grid_for(shape_for(T, P), T, kGradWgs)) * P * sizeof(float));
}

}  // namespace

}  // namespace ssm

extern "C" {

ssm_status ssm_add_norm(int64_t T, int64_t P, int32_t io, const float* r, const void* y, const float* norm_scale,
                        float eps, float* r_out, void* x, float* rinv, void* stream) {
  const ssm_status s = ssm::check_sizes(T, P);
  if (s != SSM_OK) return s;
  if (io != SSM_F32 && io != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (!abi::good(r) || !abi::good(norm_scale) || !abi::good(x) || !abi::good_or_null(y) || !abi::good_or_null(rinv) ||
      !abi::good_or_null(r_out) || (y && !r_out) || !(eps > 0.0f) || !isfinite(eps))
    return SSM_ERR_ARG;
  ssm::NormArgs a{};
  a.T = T; a.P = P; a.r = r; a.y = y; a.scale = norm_scale; a.eps = eps;
  a.r_out = (!y && r_out == r) ? nullptr : r_out;  // nothing to write
  a.x = x; a.rinv = rinv;
  return ssm::launch_norm<false>(a, io == SSM_BF16, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                                   : SSM_ERR_HIP;
}

size_t ssm_add_norm_grad_workspace_bytes(int64_t T, int64_t P) {
  return ssm::check_sizes(T, P) == SSM_OK ? ssm::grad_bytes(T, P) : 0;
}

ssm_status ssm_add_norm_grad(int64_t T, int64_t P, int32_t io, const float* r_out, const float* rinv,
                             const float* norm_scale, const void* dx, const float* dr_out, float* dr,
                             float* dnorm_scale, void* ws, size_t ws_bytes, void* stream) {
  ssm_status s = ssm::check_sizes(T, P);
  if (s != SSM_OK) return s;
  if (io != SSM_F32 && io != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (!abi::good(r_out) || !abi::good(rinv) || !abi::good(norm_scale) || !abi::good(dx) ||
      !abi::good_or_null(dr_out) || !abi::good(dr) || !abi::good_or_null(dnorm_scale))
    return SSM_ERR_ARG;
  if ((s = abi::check_ws(ws, ws_bytes, ssm::grad_bytes(T, P))) != SSM_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  ssm::NormArgs a{};
  a.T = T; a.P = P; a.r = r_out; a.rinv_in = rinv; a.scale = norm_scale; a.y = dx; a.dr_out = dr_out; a.r_out = dr;
  a.part = dnorm_scale ? static_cast<float*>(ws) : nullptr;
  if (ssm::launch_norm<true>(a, io == SSM_BF16, st) != hipSuccess) return SSM_ERR_HIP;
  if (dnorm_scale) {
    const int nb = static_cast<int>(ssm::grid_for(ssm::shape_for(T, P), T, ssm::kGradWgs));
    ssm::k_column_sums<<<static_cast<unsigned>((P + 15) / 16), 256, 0, st>>>(nb, static_cast<int>(P), a.part,
                                                                           dnorm_scale);
    if (hipGetLastError() != hipSuccess) return SSM_ERR_HIP;
  }
  return SSM_OK;
}

}  // extern "C"
