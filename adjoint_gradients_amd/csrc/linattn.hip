// linattn.hip -- the C entries of include/ssm_linattn.h: validation, the
// split of the sequences into segments, the workspace, the launches, and the
// small kernels around the chunked recurrence of linattn.inl.
//
//   forward : [segment sums -> carry between segments ->] run over segments
//   gradient: the same two steps for the state and its adjoint, then the runs
//             for dq, dv and dk; the sums over the value heads of a key head
//             and over the tokens of a fixed decay last
//   step    : one pass over the states
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/ssm_linattn.h"
#include "abi_util.hpp"
#include "linattn_seqs.hpp"
#include "ssm_common.hpp"

namespace la {

namespace {

using ssm::bf16_t;

// ---------------------------------------------------------------- carry between segments

// A sequence's segments: how many, and the slot of the first.
struct Walk {
  int nseg;
  int64_t slot0;
};

__device__ __forceinline__ Walk walk_of(const Seqs& sq, int s) {
  const uint32_t T = static_cast<uint32_t>(sq.T), L = static_cast<uint32_t>(sq.L);
  const uint32_t n = T / static_cast<uint32_t>(sq.S);
  auto start = [&](int i) -> uint32_t {
    if (!sq.start) return n * static_cast<uint32_t>(i);
    const int32_t v = sq.start[i];
    return v < 0 ? 0u : static_cast<uint32_t>(v) > T ? T : static_cast<uint32_t>(v);
  };
  const uint32_t t0 = start(s), t1 = start(s + 1);
  if (t1 <= t0) return Walk{0, 0};
  return Walk{static_cast<int>((t1 - t0 + L - 1) / L), t0 / L + static_cast<uint32_t>(s)};
}

// Turns the segments' sums into the states entering them, in place: x starts
// as the sequence's end state, seg[j] <- x, x <- decay_j x + old seg[j], over
// the segments in order (reverse: from the last).  One thread per four
// floats; the loads of up to 16 segments are in flight together.  Sequences of
// one segment have none.  Bound by the states' traffic: 32 us for 2048 states
// of 64 KB, read and written (8.4 TB/s, since the pass before left much of them
// in the caches).
struct CarryArgs {
  Seqs sq;
  int32_t Hv, dkdv, tiles;
  const float* s0[2];
  float* seg[2];
  const float* decay[2];
};

__global__ __launch_bounds__(256) void k_la_carry(CarryArgs a) {
  const bool rev = blockIdx.x >= static_cast<unsigned>(a.tiles);
  const int tile = rev ? blockIdx.x - a.tiles : blockIdx.x;
  float* const seg = a.seg[rev];
  if (!seg) return;
  const int e = (tile * 256 + threadIdx.x) * 4;
  if (e >= a.dkdv) return;
  const int h = blockIdx.y, s = blockIdx.z;
  const Walk w = walk_of(a.sq, s);
  const int nseg = w.nseg;
  if (nseg < 2) return;
  const int64_t slot0 = w.slot0;
  float4 x{0.f, 0.f, 0.f, 0.f};
  if (a.s0[rev]) x = *reinterpret_cast<const float4*>(a.s0[rev] + (static_cast<int64_t>(s) * a.Hv + h) * a.dkdv + e);
  // N segments from j0 on, their loads in flight together
  auto walk = [&](int j0, auto batch) {
    constexpr int N = decltype(batch)::value;
    float4 u[N];
    float d[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
      // the last segment of the walk has no sum: its values are not used
      const int k = j0 + i < nseg - 1 ? j0 + i : 0;
      const int64_t o = (slot0 + (rev ? nseg - 1 - k : k)) * a.Hv + h;
      u[i] = *reinterpret_cast<const float4*>(seg + o * a.dkdv + e);
      d[i] = a.decay[rev][o];
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int k = j0 + i;
      if (k < nseg) {
        const int64_t o = (slot0 + (rev ? nseg - 1 - k : k)) * a.Hv + h;
        *reinterpret_cast<float4*>(seg + o * a.dkdv + e) = x;
        x.x = fmaf(d[i], x.x, u[i].x);
        x.y = fmaf(d[i], x.y, u[i].y);
        x.z = fmaf(d[i], x.z, u[i].z);
        x.w = fmaf(d[i], x.w, u[i].w);
      }
    }
  };
  int j0 = 0;
  for (; j0 + 16 <= nseg; j0 += 16) walk(j0, std::integral_constant<int, 16>{});
  for (; j0 < nseg; j0 += 4) walk(j0, std::integral_constant<int, 4>{});
}

// The same with the walk cut into kWalks parts of a workgroup, for many
// segments of few states: each part sums its segments, takes the state that
// the parts before it leave, and walks again.  Bound by the latency of a part.
constexpr int kWalks = 16;

__global__ __launch_bounds__(256) void k_la_carry_split(CarryArgs a) {
  constexpr int kCols = 256 / kWalks;
  __shared__ float4 sums[kWalks][kCols];
  __shared__ float decays[kWalks];
  const bool rev = blockIdx.x >= static_cast<unsigned>(a.tiles);
  const int tile = rev ? blockIdx.x - a.tiles : blockIdx.x;
  float* const seg = a.seg[rev];
  if (!seg) return;
  const int h = blockIdx.y, s = blockIdx.z;
  const Walk w = walk_of(a.sq, s);
  if (w.nseg < 2) return;
  const int col = threadIdx.x % kCols, part = threadIdx.x / kCols;
  const int e = (tile * kCols + col) * 4;  // a state is a multiple of kCols * 4 floats
  const int n = (w.nseg + kWalks - 1) / kWalks;
  const int k0 = part * n, k1 = k0 + n < w.nseg ? k0 + n : w.nseg;
  auto slot = [&](int k) { return (w.slot0 + (rev ? w.nseg - 1 - k : k)) * a.Hv + h; };
  auto walk = [&](float4 x, bool put) {
    float d = 1.0f;
    for (int j0 = k0; j0 < k1; j0 += 8) {
      float4 u[8];
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        // the last segment of the sequence's walk has no sum: its values are not used
        const int k = j0 + i < k1 && j0 + i < w.nseg - 1 ? j0 + i : 0;
        u[i] = *reinterpret_cast<const float4*>(seg + slot(k) * a.dkdv + e);
        f[i] = a.decay[rev][slot(k)];
      }
#pragma unroll
      for (int i = 0; i < 8; i++) {
        if (j0 + i < k1) {
          if (put) *reinterpret_cast<float4*>(seg + slot(j0 + i) * a.dkdv + e) = x;
          x.x = fmaf(f[i], x.x, u[i].x);
          x.y = fmaf(f[i], x.y, u[i].y);
          x.z = fmaf(f[i], x.z, u[i].z);
          x.w = fmaf(f[i], x.w, u[i].w);
          d *= f[i];
        }
      }
    }
    sums[part][col] = x;
    if (col == 0) decays[part] = d;
  };
  walk(float4{0.f, 0.f, 0.f, 0.f}, false);
  __syncthreads();
  float4 x{0.f, 0.f, 0.f, 0.f};
  if (a.s0[rev]) x = *reinterpret_cast<const float4*>(a.s0[rev] + (static_cast<int64_t>(s) * a.Hv + h) * a.dkdv + e);
  for (int p = 0; p < part; p++) {
    const float4 u = sums[p][col];
    const float d = decays[p];
    x.x = fmaf(d, x.x, u.x);
    x.y = fmaf(d, x.y, u.y);
    x.z = fmaf(d, x.z, u.z);
    x.w = fmaf(d, x.w, u.w);
  }
  __syncthreads();
  walk(x, true);
}

// ---------------------------------------------------------------- sums over shared heads and tokens

// out[t][hk][c] = sum over the heads of hk's group, in order, for the rows the
// sequences cover.  One thread per four channels.  The addends stay fp32, so
// that many heads cost no digits; reading them bounds it (24 heads of 64,
// 131072 tokens, dq and dk: 1.6 GB in 387 us, 4.2 TB/s).
struct GroupArgs {
  const float* part;  // [T][Hv][d]
  void* out;          // [T][Hk][d] in the io type
};

template <class T>
__device__ __forceinline__ void group_sum(const Seqs& sq, int32_t Hk, int32_t G, int32_t d, const GroupArgs& a,
                                          int64_t wg, int64_t wgs) {
  int64_t t0 = 0, t1 = sq.T;
  if (sq.start) {
    t0 = sq.start[0];
    t1 = sq.start[sq.S];
    t0 = t0 < 0 ? 0 : t0;
    t1 = t1 > sq.T ? sq.T : t1;
  }
  const int d4 = d / 4;
  const int64_t n = t1 * Hk * d4;
  T* const out = static_cast<T*>(a.out);
  for (int64_t i = t0 * Hk * d4 + wg * 256 + threadIdx.x; i < n; i += wgs * 256) {
    const int64_t th = i / d4;
    const int c = static_cast<int>(i % d4) * 4;
    const float* p = a.part + th * G * d + c;
    float4 s = *reinterpret_cast<const float4*>(p);
    for (int g = 1; g < G; g++) {
      const float4 v = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(g) * d);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    T* o = out + th * d + c;
    ssm::store_io(o, s.x); ssm::store_io(o + 1, s.y); ssm::store_io(o + 2, s.z); ssm::store_io(o + 3, s.w);
  }
}

// The decay gradient from the runs' terms, one workgroup per segment and
// head: for the chunks of each anchor, from the last,
//   dg_t = (sum over i >= t, forward run) + (sum over j < t, reverse run) + x_c,
// x_c = e^{G_L} <S, D> at the anchor; then x of the chunk before is x_c plus
// c's sum over all i less its own sum over all j.  Bound by the kept states:
// 68 us for 2 x 2048 of 64 KB (3.9 TB/s).
struct DecayArgs {
  Seqs sq;
  int32_t Hv, ch, n4;           // tokens of a chunk; float4s of a padded state
  const float* log_decay;
  int64_t ld_decay;
  const float *tok_f, *tok_r;   // [Hv][T]
  const float *anchor_s, *anchor_d;
  float* dg_tok;                // [T][Hv] or null
  double* dg_seg;               // [slots][Hv] or null
};

__device__ __forceinline__ double wg_sum(double v, double* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__device__ __forceinline__ void decay_grad(const DecayArgs& a, uint32_t slot, int h) {
  __shared__ double red[4], xs[kAnchor], all_i[kAnchor], all_j[kAnchor];
  Segment sg;
  const bool have = find_segment(a.sq, slot, a.ch, &sg);
  double sum = 0.0;
  if (have) {
    const int nch = (sg.t1 - sg.t0 + a.ch - 1) / a.ch;
    const float* const tf = a.tok_f + static_cast<int64_t>(h) * a.sq.T;
    const float* const tr = a.tok_r + static_cast<int64_t>(h) * a.sq.T;
    for (int k0 = 0; k0 < nch; k0 += kAnchor) {
      const int c = nch - 1 - k0;  // the anchor
      const int nc = c + 1 < kAnchor ? c + 1 : kAnchor;
      const int64_t o = ((anchor_slot(sg, slot) + k0 / kAnchor) * a.Hv + h) * a.n4;
      const float4* const ps = reinterpret_cast<const float4*>(a.anchor_s) + o;
      const float4* const pd = reinterpret_cast<const float4*>(a.anchor_d) + o;
      double dot = 0.0;
#pragma unroll 4
      for (int i = threadIdx.x; i < a.n4; i += 256) {
        const float4 s = ps[i], d = pd[i];
        dot += static_cast<double>(fmaf(s.x, d.x, s.y * d.y) + fmaf(s.z, d.z, s.w * d.w));
      }
      const int t = sg.t0 + c * a.ch + static_cast<int>(threadIdx.x);
      double lg = 0.0;
      if (static_cast<int>(threadIdx.x) < a.ch && t < sg.t1)
        lg = decay_log2(a.log_decay[t * a.ld_decay + h]);
      lg = wg_sum(lg, red);
      dot = wg_sum(dot, red);
      // sums of chunk c - i over all its tokens, for the boundary on either side
      if (static_cast<int>(threadIdx.x) < nc) {
        const int first = sg.t0 + (c - static_cast<int>(threadIdx.x)) * a.ch;
        const int end = first + a.ch < sg.t1 ? first + a.ch : sg.t1;
        all_i[threadIdx.x] = static_cast<double>(tf[first]);
        all_j[threadIdx.x] = static_cast<double>(tr[end - 1]);
      }
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < nc) {
        double x = static_cast<double>(exp2_split(lg)) * dot;
        for (int i = 0; i < static_cast<int>(threadIdx.x); i++) x += all_i[i] - all_j[i + 1];
        xs[threadIdx.x] = x;
      }
      __syncthreads();
      const int t0 = sg.t0 + (c + 1 - nc) * a.ch;
      const int t1 = sg.t0 + (c + 1) * a.ch < sg.t1 ? sg.t0 + (c + 1) * a.ch : sg.t1;
      for (int u = t0 + static_cast<int>(threadIdx.x); u < t1; u += 256) {
        const int j = (u - sg.t0) / a.ch;
        const double before = u == sg.t0 + j * a.ch ? 0.0 : static_cast<double>(tr[u - 1]);
        const double dg = static_cast<double>(tf[u]) + before + xs[c - j];
        if (a.dg_tok) a.dg_tok[static_cast<int64_t>(u) * a.Hv + h] = static_cast<float>(dg);
        sum += dg;
      }
      __syncthreads();
    }
  }
  if (a.dg_seg) {
    sum = wg_sum(sum, red);
    if (threadIdx.x == 0) a.dg_seg[static_cast<int64_t>(slot) * a.Hv + h] = sum;
  }
}

// What follows the runs of the gradient, in one launch: first the workgroups
// of the decay gradient (decay_wgs of them), then those of the sums of dq and
// of dk over shared heads (sum_wgs each).
struct FinishArgs {
  DecayArgs decay;
  GroupArgs group[2];
  int32_t Hk, dk;
  uint32_t decay_wgs, sum_wgs;
};

template <class T>
__global__ __launch_bounds__(256) void k_la_finish(FinishArgs a) {
  const uint32_t b = blockIdx.x;
  if (b < a.decay_wgs) {
    decay_grad(a.decay, b / a.decay.Hv, static_cast<int>(b % a.decay.Hv));
    return;
  }
  const uint32_t k = b - a.decay_wgs;
  group_sum<T>(a.decay.sq, a.Hk, a.decay.Hv / a.Hk, a.dk, a.group[k / a.sum_wgs], k % a.sum_wgs, a.sum_wgs);
}

// out[h] = sum over the segments, in a fixed order, in 64 bits.
__global__ __launch_bounds__(256) void k_la_decay_sum(int64_t slots, int32_t Hv, const double* __restrict__ part,
                                                     float* __restrict__ out) {
  __shared__ double red[256];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < slots; i += 256) s += part[i * Hv + h];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int d = 128; d >= 1; d >>= 1) {
    if (threadIdx.x < static_cast<unsigned>(d)) red[threadIdx.x] += red[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x == 0) out[h] = static_cast<float>(red[0]);
}

// ---------------------------------------------------------------- single tokens

// h <- e^g h + k v^T, y = scale q h for one row and head and NC of the dv
// columns per workgroup.  The state is read and written once, 16 bytes a
// lane; a column of lanes strides the dk rows and their partial sums of y
// meet in LDS.  Bound by the state's traffic: 192 rows of 16 heads of 128, 76 us
// (5.3 TB/s).  STREAM: past the caches, for states that they will not hold
// until the next token.
struct StepArgs {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv, ldy;
  const float* log_decay;
  int64_t ld_decay;
  float* state;
  void* y;
  int32_t Hv, G, dk, dv, tiles;
  float scale;
};

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;

template <bool STREAM>
__device__ __forceinline__ float4 state_load(const float* p) {
  const f32x4* const v = reinterpret_cast<const f32x4*>(p);
  return __builtin_bit_cast(float4, STREAM ? __builtin_nontemporal_load(v) : *v);
}
template <bool STREAM>
__device__ __forceinline__ void state_store(float* p, float4 x) {
  f32x4* const v = reinterpret_cast<f32x4*>(p);
  if (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(f32x4, x), v);
  else *v = __builtin_bit_cast(f32x4, x);
}

template <class T, int NC, bool STREAM>
__global__ __launch_bounds__(256) void k_la_step(StepArgs a) {
  constexpr int CG = NC / 4;        // lanes across the columns
  constexpr int RG = 256 / CG;      // lanes down the rows
  constexpr int NR = 128 / RG;      // rows a lane, at most
  __shared__ float sq[128], sk[128];
  __shared__ float4 red[RG][CG];
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y / a.tiles, c0 = blockIdx.y % a.tiles * NC;
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
  const int c = c0 + 4 * cg;
  const bool in = c < a.dv;
  float* const st = a.state + ((t * a.Hv + h) * a.dk) * a.dv + c;
  float4 s[NR];
#pragma unroll
  for (int i = 0; i < NR; i++) {
    const int m = rg + RG * i;
    if (in && m < a.dk) s[i] = state_load<STREAM>(st + m * a.dv);
  }
  const int hk = h / a.G;
  if (threadIdx.x < static_cast<unsigned>(a.dk)) {
    sq[threadIdx.x] = ssm::load_io(static_cast<const T*>(a.q) + t * a.ldq + hk * a.dk + threadIdx.x) * a.scale;
    sk[threadIdx.x] = ssm::load_io(static_cast<const T*>(a.k) + t * a.ldk + hk * a.dk + threadIdx.x);
  }
  float4 v{0.f, 0.f, 0.f, 0.f};
  if (in) {
    const T* p = static_cast<const T*>(a.v) + t * a.ldv + h * a.dv + c;
    v = float4{ssm::load_io(p), ssm::load_io(p + 1), ssm::load_io(p + 2), ssm::load_io(p + 3)};
  }
  // e^g with g log2 e in two floats, so that a strong decay keeps its digits
  const double g2 = static_cast<double>(a.log_decay[t * a.ld_decay + h]) * 1.4426950408889634;
  const float gh = static_cast<float>(g2);
  const float gl = gh < -16000.0f ? 0.0f : static_cast<float>(g2 - static_cast<double>(gh));
  const float e = ssm::fast_exp2(gh);
  const float w = fmaf(e, gl * 0.69314718055994531f, e);
  __syncthreads();
  float4 y{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NR; i++) {
    const int m = rg + RG * i;
    if (in && m < a.dk) {
      const float k = sk[m], q = sq[m];
      s[i].x = fmaf(w, s[i].x, k * v.x);
      s[i].y = fmaf(w, s[i].y, k * v.y);
      s[i].z = fmaf(w, s[i].z, k * v.z);
      s[i].w = fmaf(w, s[i].w, k * v.w);
      state_store<STREAM>(st + m * a.dv, s[i]);
      y.x = fmaf(q, s[i].x, y.x);
      y.y = fmaf(q, s[i].y, y.y);
      y.z = fmaf(q, s[i].z, y.z);
      y.w = fmaf(q, s[i].w, y.w);
    }
  }
  red[rg][cg] = y;
  __syncthreads();
  if (rg == 0 && in) {
    for (int i = 1; i < RG; i++) {
      const float4 p = red[i][cg];
      y.x += p.x; y.y += p.y; y.z += p.z; y.w += p.w;
    }
    T* o = static_cast<T*>(a.y) + t * a.ldy + h * a.dv + c;
    ssm::store_io(o, y.x); ssm::store_io(o + 1, y.y); ssm::store_io(o + 2, y.z); ssm::store_io(o + 3, y.w);
  }
}

// ---------------------------------------------------------------- host side

using abi::good;
using abi::good_or_null;

constexpr int32_t kMaxHeads = 4096, kMaxSeqs = 65535;
constexpr int64_t kMaxSeqHeads = int64_t(1) << 22;  // three runs of them are a grid's limit of 2^32 lanes
constexpr int64_t kMaxLd = int64_t(1) << 22;  // a chunk's rows stay within 32-bit byte offsets
constexpr int64_t kMaxStepRows = int64_t(1) << 22;

size_t es(const ssm_linattn_dims* d) { return d->io == SSM_BF16 ? 2 : 4; }

ssm_status check_dims(const ssm_linattn_dims* d) {
  if (!d) return SSM_ERR_ARG;
  if (d->T < 1 || d->S < 1 || d->Hk < 1 || d->Hv < 1 || d->dk < 1 || d->dv < 1) return SSM_ERR_ARG;
  if (d->Hv % d->Hk != 0 || !isfinite(d->scale) || (d->decay_tokens != 0 && d->decay_tokens != 1)) return SSM_ERR_ARG;
  if (d->io != SSM_F32 && d->io != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (d->dk % 8 || d->dv % 8 || d->dk > 128 || d->dv > 128) return SSM_ERR_UNSUPPORTED;
  if (d->Hv > kMaxHeads || d->S > kMaxSeqs || d->T > INT32_MAX) return SSM_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->S) * d->Hv > kMaxSeqHeads) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

bool good_ld(const ssm_linattn_dims* d, int64_t ld, int64_t row) {
  return ld >= row && (ld * static_cast<int64_t>(es(d))) % 16 == 0 && ld <= kMaxLd;
}

ssm_status check_in(const ssm_linattn_dims* d, const ssm_linattn_in* in) {
  if (!in || !good(in->q) || !good(in->k) || !good(in->v) || !good(in->log_decay)) return SSM_ERR_ARG;
  if (!good_or_null(in->seq_start) || !good_or_null(in->h0)) return SSM_ERR_ARG;
  const int64_t rk = static_cast<int64_t>(d->Hk) * d->dk, rv = static_cast<int64_t>(d->Hv) * d->dv;
  if (!good_ld(d, in->ldq, rk) || !good_ld(d, in->ldk, rk) || !good_ld(d, in->ldv, rv)) return SSM_ERR_ARG;
  return SSM_OK;
}

// Tokens per segment.  A run walks its segment chunk by chunk, and a segment
// costs one more read of two of its operands and two passes over a state.
// With much work a segment is a quarter of what a workgroup would have if all
// of them ran at once (kRounds: some XCDs are a sixth slower, and the later
// rounds even that out), of at least kChunks chunks; with little, it is as
// short as still gives every place on the chip one, down to kMinChunks.
// Gradient of 65536 tokens, 16 heads of 128: 1.78, 1.62, 1.52, 1.53 ms with 1,
// 2, 4, 8 rounds.  8192 tokens: 271, 245, 214, 258 us with segments of 2, 4,
// 8, 16 chunks; forward of 2048 tokens: 36, 40, 60, 105 us.
constexpr int64_t kCus = 256;
constexpr int64_t kRounds = 4;
constexpr int64_t kChunks = 8, kMinChunks = 2;

int64_t longest(const ssm_linattn_dims* d, bool packed) { return packed ? d->T : d->T / d->S; }

int64_t segment_tokens(const ssm_linattn_dims* d, bool packed, int runs) {
  const int64_t ch = chunk_tokens(d->io == SSM_BF16);
  const int64_t places = kCus * (padded(d->dk) * padded(d->dv) > 64 * 64 ? 2 : 3);
  const int64_t work = d->T * d->Hv * runs / ch;  // chunks of all heads and runs
  const int64_t one_round = (work + places - 1) / places;
  int64_t chunks = one_round < kMinChunks ? kMinChunks : one_round < kChunks ? one_round : kChunks;
  if (chunks < work / (places * kRounds)) chunks = work / (places * kRounds);
  const int64_t L = chunks * ch;
  const int64_t n = (longest(d, packed) + ch - 1) / ch * ch;
  return L < n ? L : n;
}

struct Ws {
  float* seg[2];        // segment states: forward, adjoint
  float* seg_decay[2];
  float* tok[2];        // the decay gradient's terms: forward run, reverse run
  float* anchors[2];
  double* dg_seg;
  float* part[2];       // dq, dk per value head
};

struct Plan {
  int64_t L, slots;
  bool split;           // some sequence may have several segments
  bool need_s, need_d;  // the runs that use the state / its adjoint
  bool dg;
};

// Packed sequences may be any length up to T, so the plan covers both forms
// of the sequences with the same sizes: what a caller asks for with
// ssm_linattn_workspace_bytes does not depend on seq_start.
Plan make_plan(const ssm_linattn_dims* d, const ssm_linattn_grads* g, bool packed) {
  Plan p{};
  p.need_s = !g || g->dq || g->dlog_decay;
  p.need_d = g && (g->dk || g->dv || g->dlog_decay || g->dh0);
  p.dg = g && g->dlog_decay;
  p.L = segment_tokens(d, packed, g ? 3 : 1);
  p.slots = slot_count(d->T, d->S, p.L);
  p.split = p.L < longest(d, packed);
  return p;
}

Ws carve(abi::Carver& cv, const ssm_linattn_dims* d, const ssm_linattn_grads* g, const Plan& p) {
  Ws w{};
  const size_t hs = static_cast<size_t>(p.slots) * d->Hv;
  if (p.split) {
    const bool need[2] = {p.need_s, p.need_d};
    for (int i = 0; i < 2; i++)
      if (need[i]) {
        w.seg[i] = cv.take<float>(hs * d->dk * d->dv);
        w.seg_decay[i] = cv.take<float>(hs);
      }
  }
  if (p.dg) {
    // chunk slots of consecutive segments are kAnchor apart at least where their anchors are
    const int64_t n = slot_count(d->T, d->S, chunk_tokens(d->io == SSM_BF16)) / kAnchor + p.slots + 1;
    for (int i = 0; i < 2; i++) {
      w.tok[i] = cv.take<float>(static_cast<size_t>(d->T) * d->Hv);
      w.anchors[i] = cv.take<float>(static_cast<size_t>(n) * d->Hv * state_floats(d->dk, d->dv));
    }
    if (!d->decay_tokens) w.dg_seg = cv.take<double>(hs);
  }
  if (g && d->Hk != d->Hv) {
    const void* outs[2] = {g->dq, g->dk};
    for (int i = 0; i < 2; i++)
      if (outs[i]) w.part[i] = cv.take<float>(static_cast<size_t>(d->T) * d->Hv * d->dk);
  }
  return w;
}

size_t plan_bytes(const ssm_linattn_dims* d, const ssm_linattn_grads* g) {
  size_t most = 0;
  for (int packed = 0; packed < 2; packed++) {
    abi::Carver cv(nullptr);
    carve(cv, d, g, make_plan(d, g, packed != 0));
    if (cv.off > most) most = cv.off;
  }
  return most;
}

bool any_grad(const ssm_linattn_grads* g) { return g->dq || g->dk || g->dv || g->dlog_decay || g->dh0; }

// Launches the runs of a kernel that have operands.
hipError_t launch(Kernel k, const ssm_linattn_dims* d, Args& a, hipStream_t st) {
  a.nz = 0;
  for (int i = 0; i < 3; i++)
    if (a.run[i].K) a.run_of[a.nz++] = i;
  a.units = static_cast<uint32_t>(slot_count(d->T, d->S, a.sq.L) * d->Hv);
  const bool wide = padded(d->dk) == 128;
  if (d->io == SSM_BF16) return wide ? launch_bf16_128(k, d->dv, a, st) : launch_bf16_64(k, d->dv, a, st);
  return wide ? launch_f32_128(k, d->dv, a, st) : launch_f32_64(k, d->dv, a, st);
}

Args base_args(const ssm_linattn_dims* d, const ssm_linattn_in* in, const Plan& p) {
  Args a{};
  a.sq = Seqs{d->T, d->S, in->seq_start, p.L};
  a.Hv = d->Hv;
  a.dkdv = d->dk * d->dv;
  a.log_decay = in->log_decay;
  a.ld_decay = d->decay_tokens ? d->Hv : 0;
  a.sum_heads = d->Hk != d->Hv;
  return a;
}

// An operand of a run: token rows with G value heads per head.
struct Op {
  const void* p;
  int64_t ld;
  int32_t g, d;
};

Run make_run(const Op& q, const Op& k, const Op& v, float qs, float ks) {
  Run r{};
  r.Q = q.p; r.ldq = q.ld; r.gq = q.g;
  r.K = k.p; r.ldk = k.ld; r.gk = k.g;
  r.V = v.p; r.ldv = v.ld; r.gv = v.g;
  r.dm = k.d; r.dn = v.d;
  r.qs = qs; r.ks = ks;
  return r;
}

// The segments' entering states, for the directions in use (runs of the aggregate kernel).
hipError_t carry_states(Kernel sums, const ssm_linattn_dims* d, Args a, const Run& fwd, const Run& rev, const Ws& w,
                        const float* h0, const float* dhT, hipStream_t st) {
  a.run[0] = fwd;
  a.run[1] = rev;
  for (int i = 0; i < 2; i++) {
    a.run[i].seg = w.seg[i];
    a.run[i].seg_decay = w.seg_decay[i];
    a.run[i].sm = d->dv;
    a.run[i].sn = 1;
  }
  hipError_t e = launch(sums, d, a, st);
  if (e != hipSuccess) return e;
  CarryArgs c{};
  c.sq = a.sq;
  c.Hv = d->Hv;
  c.dkdv = a.dkdv;
  // Long walks of few states leave the chip idle unless they are cut; with
  // many states the second read costs more.  Forward, whole and cut: 65536
  // tokens, 1, 4, 16 heads of 128: 113, 150, 497 us and 60, 124, 497; 131072
  // tokens, 1, 4, 24 heads of 64: 124, 127, 652 and 49, 102, 650; 4096 tokens,
  // 16 heads of 128: 58 and 65; 16 or 8 segments, 4 heads of 64: 17.7 and 17.7,
  // 16.4 and 17.0.
  const int64_t tiles = (a.dkdv / 4 + 255) / 256;
  const int64_t most = (longest(d, a.sq.start != nullptr) + a.sq.L - 1) / a.sq.L;
  const bool split = most > kWalks && tiles * d->Hv * d->S <= 64;
  c.tiles = static_cast<int32_t>(split ? a.dkdv / 4 / (256 / kWalks) : tiles);
  c.s0[0] = h0; c.s0[1] = dhT;
  for (int i = 0; i < 2; i++) {
    c.seg[i] = w.seg[i];
    c.decay[i] = w.seg_decay[i];
  }
  const dim3 grid(static_cast<unsigned>(c.tiles * (w.seg[1] ? 2 : 1)), static_cast<unsigned>(d->Hv),
                  static_cast<unsigned>(d->S));
  if (split) k_la_carry_split<<<grid, 256, 0, st>>>(c);
  else k_la_carry<<<grid, 256, 0, st>>>(c);
  return hipGetLastError();
}

hipError_t run_forward(const ssm_linattn_dims* d, const ssm_linattn_in* in, void* y, int64_t ldy, float* hT, void* ws,
                       hipStream_t st) {
  const Plan p = make_plan(d, nullptr, in->seq_start != nullptr);
  abi::Carver cv(ws);
  const Ws w = carve(cv, d, nullptr, p);
  const int32_t G = d->Hv / d->Hk;
  const Op q{in->q, in->ldq, G, d->dk}, k{in->k, in->ldk, G, d->dk}, v{in->v, in->ldv, 1, d->dv};
  Args a = base_args(d, in, p);
  Run r = make_run(q, k, v, d->scale, 1.0f);
  if (p.split) {
    hipError_t e = carry_states(hT ? kAggregate : kAggregateOut, d, a, r, Run{}, w, in->h0, nullptr, st);
    if (e != hipSuccess) return e;
  }
  r.s0 = in->h0;
  r.seg = w.seg[0];
  r.s_end = hT;
  r.sm = d->dv;
  r.sn = 1;
  r.out = y;
  r.ldo = ldy;
  a.run[0] = r;
  return launch(hT ? kForwardState : kForward, d, a, st);
}

hipError_t run_grad(const ssm_linattn_dims* d, const ssm_linattn_in* in, const void* dy, int64_t lddy,
                    const float* dhT, const ssm_linattn_grads* g, void* ws, hipStream_t st) {
  const Plan p = make_plan(d, g, in->seq_start != nullptr);
  abi::Carver cv(ws);
  const Ws w = carve(cv, d, g, p);
  const int32_t G = d->Hv / d->Hk;
  const Op q{in->q, in->ldq, G, d->dk}, k{in->k, in->ldk, G, d->dk}, v{in->v, in->ldv, 1, d->dv},
      o{dy, lddy, 1, d->dv};
  Args a = base_args(d, in, p);
  hipError_t e;
  if (p.split) {
    const Run fwd = p.need_s ? make_run(k, k, v, 1.0f, 1.0f) : Run{};
    const Run rev = p.need_d ? make_run(q, q, o, 1.0f, d->scale) : Run{};
    const Kernel sums = p.dg || g->dh0 ? kAggregate : kAggregateOut;
    if ((e = carry_states(sums, d, a, fwd, rev, w, in->h0, dhT, st)) != hipSuccess) return e;
  }
  const int64_t part_ld = static_cast<int64_t>(d->Hv) * d->dk;
  // dq: state S^T, entered by h0
  Run rq = make_run(o, v, k, d->scale, 1.0f);
  rq.X = q.p; rq.ldx = q.ld;
  rq.s0 = in->h0;
  rq.seg = w.seg[0];
  rq.sm = 1; rq.sn = d->dv;
  rq.out = w.part[0] ? static_cast<void*>(w.part[0]) : g->dq;
  rq.ldo = part_ld;
  rq.tok = w.tok[0];
  rq.anchors = w.anchors[0];
  // dv: the state's adjoint D, entered by dhT
  Run rv = make_run(k, q, o, 1.0f, d->scale);
  rv.s0 = dhT;
  rv.seg = w.seg[1];
  rv.sm = d->dv; rv.sn = 1;
  rv.out = g->dv;
  rv.ldo = static_cast<int64_t>(d->Hv) * d->dv;
  // dk: D^T
  Run rk = make_run(v, o, q, 1.0f, d->scale);
  rk.X = k.p; rk.ldx = k.ld;
  rk.s0 = dhT;
  rk.seg = w.seg[1];
  rk.sm = 1; rk.sn = d->dv;
  rk.out = w.part[1] ? static_cast<void*>(w.part[1]) : g->dk;
  rk.ldo = part_ld;
  rk.tok = w.tok[1];
  rk.anchors = w.anchors[1];
  const bool need_k = g->dk || g->dh0 || p.dg;
  rk.s_end = g->dh0;
  a.run[0] = g->dq || p.dg ? rq : Run{};
  a.run[1] = need_k ? rk : Run{};
  a.run[2] = g->dv ? rv : Run{};
  if ((e = launch(p.dg ? kGradDecay : kGradPlain, d, a, st)) != hipSuccess) return e;
  FinishArgs f{};
  f.decay.sq = a.sq;
  f.decay.Hv = d->Hv;
  f.Hk = d->Hk;
  f.dk = d->dk;
  if (p.dg) {
    f.decay = DecayArgs{a.sq, d->Hv, chunk_tokens(d->io == SSM_BF16),
                        static_cast<int32_t>(state_floats(d->dk, d->dv) / 4), in->log_decay, a.ld_decay, w.tok[0],
                        w.tok[1], w.anchors[0], w.anchors[1], d->decay_tokens ? g->dlog_decay : nullptr, w.dg_seg};
    f.decay_wgs = static_cast<uint32_t>(p.slots * d->Hv);
  }
  uint32_t sums = 0;
  for (int i = 0; i < 2; i++)
    if (w.part[i]) f.group[sums++] = GroupArgs{w.part[i], i == 0 ? g->dq : g->dk};
  if (sums) {
    const int64_t wgs = (d->T * d->Hk * (d->dk / 4) + 255) / 256;
    f.sum_wgs = static_cast<uint32_t>(wgs < 2048 ? wgs : 2048);
  }
  const uint32_t grid = f.decay_wgs + sums * f.sum_wgs;
  if (grid) {
    if (d->io == SSM_BF16) k_la_finish<bf16_t><<<grid, 256, 0, st>>>(f);
    else k_la_finish<float><<<grid, 256, 0, st>>>(f);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (w.dg_seg) {
    k_la_decay_sum<<<static_cast<unsigned>(d->Hv), 256, 0, st>>>(p.slots, d->Hv, w.dg_seg, g->dlog_decay);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class T>
hipError_t run_step(StepArgs a, int64_t rows, hipStream_t st) {
  // Narrow column tiles while the whole-row form would leave CUs idle: 16, 64,
  // 256 rows and heads take 3.7, 4.1, 7.1 us in tiles, 5.9, 6.2, 8.1 whole; 512
  // and 1024 take 9.9, 22.4 in tiles, 10.1, 21.3 whole.
  const bool narrow = rows * a.Hv < 512;
  a.tiles = narrow ? (a.dv + 31) / 32 : 1;
  const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(a.Hv * a.tiles));
  // From a quarter of the 256 MB cache on, the states of a few layers evict one
  // another.  Five of them in turn, 16 heads of 128, cached and streamed: 192
  // rows 87 and 76 us, 64 rows (67 MB) 35 and 26, 32 rows 13.4 and 13.9; one
  // alone: 60 and 75, 21.5 and 22.8, 9.9 and 11.8.
  const bool stream = rows * a.Hv * a.dk * a.dv * 4 >= (int64_t(64) << 20);
  if (narrow) k_la_step<T, 32, false><<<grid, 256, 0, st>>>(a);
  else if (stream) k_la_step<T, 128, true><<<grid, 256, 0, st>>>(a);
  else k_la_step<T, 128, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

}  // namespace la

// ---------------------------------------------------------------- C entries

extern "C" {

ssm_status ssm_linattn_workspace_bytes(const ssm_linattn_dims* dims, const ssm_linattn_grads* grads, size_t* bytes) {
  if (!bytes) return SSM_ERR_ARG;
  *bytes = 0;
  const ssm_status s = la::check_dims(dims);
  if (s != SSM_OK) return s;
  if (grads && !la::any_grad(grads)) return SSM_ERR_ARG;
  *bytes = la::plan_bytes(dims, grads);
  return SSM_OK;
}

ssm_status ssm_linattn_forward(const ssm_linattn_dims* dims, const ssm_linattn_in* in, void* y, int64_t ldy, float* hT,
                               void* ws, size_t ws_bytes, void* stream) {
  ssm_status s = la::check_dims(dims);
  if (s != SSM_OK) return s;
  if ((s = la::check_in(dims, in)) != SSM_OK) return s;
  if (!in->seq_start && dims->T % dims->S != 0) return SSM_ERR_ARG;
  if (!abi::good(y) || !abi::good_or_null(hT)) return SSM_ERR_ARG;
  if (!la::good_ld(dims, ldy, static_cast<int64_t>(dims->Hv) * dims->dv)) return SSM_ERR_ARG;
  if ((s = abi::check_ws(ws, ws_bytes, la::plan_bytes(dims, nullptr))) != SSM_OK) return s;
  return la::run_forward(dims, in, y, ldy, hT, ws, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK
                                                                                                  : SSM_ERR_HIP;
}

ssm_status ssm_linattn_grad(const ssm_linattn_dims* dims, const ssm_linattn_in* in, const void* dy, int64_t lddy,
                            const float* dhT, const ssm_linattn_grads* grads, void* ws, size_t ws_bytes, void* stream) {
  ssm_status s = la::check_dims(dims);
  if (s != SSM_OK) return s;
  if ((s = la::check_in(dims, in)) != SSM_OK) return s;
  if (!in->seq_start && dims->T % dims->S != 0) return SSM_ERR_ARG;
  if (!abi::good(dy) || !abi::good_or_null(dhT) || !grads || !la::any_grad(grads)) return SSM_ERR_ARG;
  if (!la::good_ld(dims, lddy, static_cast<int64_t>(dims->Hv) * dims->dv)) return SSM_ERR_ARG;
  const void* outs[] = {grads->dq, grads->dk, grads->dv, grads->dlog_decay, grads->dh0};
  for (const void* o : outs)
    if (!abi::good_or_null(o)) return SSM_ERR_ARG;
  if ((s = abi::check_ws(ws, ws_bytes, la::plan_bytes(dims, grads))) != SSM_OK) return s;
  return la::run_grad(dims, in, dy, lddy, dhT, grads, ws, static_cast<hipStream_t>(stream)) == hipSuccess
             ? SSM_OK
             : SSM_ERR_HIP;
}

ssm_status ssm_linattn_step(const ssm_linattn_dims* dims, const ssm_linattn_in* in, float* state, void* y, int64_t ldy,
                            void* stream) {
  if (!dims) return SSM_ERR_ARG;
  ssm_linattn_dims d = *dims;
  d.S = 1;
  ssm_status s = la::check_dims(&d);
  if (s != SSM_OK) return s;
  if (d.T > la::kMaxStepRows) return SSM_ERR_UNSUPPORTED;
  if ((s = la::check_in(&d, in)) != SSM_OK) return s;
  if (in->seq_start || in->h0 || !abi::good(state) || !abi::good(y)) return SSM_ERR_ARG;
  if (!la::good_ld(&d, ldy, static_cast<int64_t>(d.Hv) * d.dv)) return SSM_ERR_ARG;
  la::StepArgs a{in->q, in->k, in->v, in->ldq, in->ldk, in->ldv, ldy, in->log_decay, d.decay_tokens ? d.Hv : 0,
                 state, y, d.Hv, d.Hv / d.Hk, d.dk, d.dv, 1, d.scale};
  hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = d.io == SSM_BF16 ? la::run_step<ssm::bf16_t>(a, d.T, st) : la::run_step<float>(a, d.T, st);
  return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
