// linattn.inl -- chunked linear attention with a decay for each head on MFMA
// (included by the linattn_*.hip files, one per io type and width of dk).
//
// One recurrence runs everything.  For a chunk of C tokens with the
// inclusive sums G_i of the log decays inside it, the state S entering it and
// operands Q, K, V:
//   out_i = qs (e^{G_i} Q_i S + ks sum_{j <= i} e^{G_i - G_j} (Q_i . K_j) V_j)
//   S    <- e^{G_L} S + ks sum_j e^{G_L - G_j} K_j V_j^T
// and, walking the chunks in reverse (the adjoint of the state),
//   out_j = qs (e^{G_L - G_j} Q_j D + ks sum_{i >= j} e^{G_i - G_j} (Q_j . K_i) V_i)
//   D    <- e^{G_L} D + ks sum_i e^{G_i} K_i V_i^T.
// With (Q, K, V) = (q, k, v) forward this is y; the gradient is the same
// recurrence three times: dq from (dy, v, k) forward (state S^T), dv from
// (k, q, dy) and dk from (v, dy, q) in reverse (states D, D^T).
//
// Decay gradient: what passes from a token j < t to a token i >= t.  With
// M_ij = scale e^{G_i - G_j} (q_i . k_j)(dy_i . v_j), R_i = q_i . (the state's
// part of dq_i), K_j = k_j . (the state's part of dk_j):
//   dg_t = sum_{j < t <= i} M_ij + sum_{i >= t} R_i + sum_{j < t} K_j + e^{G_L} <S, D>.
// Nothing in it cancels; the shorter identity, the suffix sum over the whole
// sequence of <q, dq> - <k, dk>, loses three digits over 65536 tokens.  The
// term e^{G_L} <S, D> is formed where both runs keep their state, at every
// kAnchor-th chunk, and carried to the chunks between: across a boundary
// e^{G_L} <S, D> of the later chunk + its sum of R = that of the earlier one
// + its sum of K.  (Kept at every chunk, the states were 40% of the traffic.)
//
// One workgroup of four wavefronts walks the chunks of one segment of one
// sequence for one head.  The state stays in the accumulators of v_mfma
// 16x16 tiles, each wavefront holding all dm rows of its quarter of the dn
// columns; as laid out there it is itself the operand of Q S, with the rows
// of Q read in the matching order, so it never passes through LDS.  Q, K, V
// go through LDS; the next chunk's tiles are loaded into registers while the
// current one is computed.
//
// What bounds it (bf16, 65536 tokens, 16 heads of 128): the pass that sums the
// segments runs at memory speed (forward 131 us for 0.54 GB of k and v and
// 0.13 GB of states), the forward run nearly so (270 us for 1.07 GB of rows).
// The gradient's three runs (1.19 ms, half of it what their 3 GB would take)
// are bound by the chain scores - state - product - update of a chunk, which
// two workgroups a CU hide in part: the matrix units do 0.56 PFLOP/s, half of
// what a large library product reaches.  64-wide heads (24 of them, 131072
// tokens, one head of q and k: 124 us and 325 us for 0.40 and 0.81 GB) are
// bound by the same chain, with vector instructions busy two fifths of the time.
//
// Rounding: products are bf16 x bf16 summed in fp32 (or fp32 throughout).  An
// fp32 operand of one (the decayed scores, the state, the weighted V) is
// split into bf16 parts: two where the product only reaches bf16 outputs, so
// that their own rounding is all they are off by; three, which hold it whole,
// where it ends in an fp32 output (states, decay gradient).  With one part a
// few tokens, whose sums do not average the roundings, were off by up to 3.5e-3
// where the output's rounding is 1.5e-3; the second part costs the forward
// pass of 65536 tokens, 16 heads of 128, 2% (475 -> 484 us), its gradient 2%.
// Three parts in the segments' sums where two do: 590 us against 556 for 131072
// tokens, 24 heads of 64.
#include "linattn_seqs.hpp"
#include "ssm_common.hpp"

namespace la {

namespace {

using ssm::bf16_t;
using ssm::bf16x8_t;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4_t;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kThreads = 256;  // four wavefronts

// Modes of a run.
constexpr int kOut = 0;       // out
constexpr int kAgg = 1;       // only the state's sum over the segment
constexpr int kOutFwdDg = 2;  // out, the decay gradient's terms of the pairs that end here, the anchor states
constexpr int kOutRevDg = 3;  // out, the terms of the pairs that start here, the anchor states' adjoints

// bf16 parts of an fp32 operand of a product: three hold all 24 bits, for an
// fp32 output; two, off by 2^-17, for a bf16 one.
constexpr int kParts = 3, kOutParts = 2;

template <class T>
struct Cfg {
  static constexpr bool kBf = sizeof(T) == 2;
  static constexpr int CH = chunk_tokens(kBf);
  static constexpr int NIB = CH / 16;      // 16-token blocks
  static constexpr int JW = 4 / NIB;       // wavefronts sharing a row block of the scores
  static constexpr int EPV = 16 / sizeof(T);
  static constexpr int kPad = kBf ? 16 : 4;  // elements between the rows of a tile (see at())
};

// LDS of a run, in bytes.
template <class T, int DM, int DN, int MODE>
struct Lds {
  using C = Cfg<T>;
  static constexpr int PM = DM + C::kPad, PN = DN + C::kPad;
  static constexpr int q = 0;
  static constexpr int k = q + (MODE == kAgg ? 0 : C::CH * PM * (int)sizeof(T));
  static constexpr int v = k + C::CH * PM * (int)sizeof(T);
  static constexpr int p = v + C::CH * PN * (int)sizeof(T);
  static constexpr int f = p + (MODE == kAgg ? 0 : C::CH * C::CH * (int)sizeof(T) * (C::kBf ? kOutParts : 1));
  // Two buffers of wc in the padding of V's last row: 16 bytes more, and three
  // workgroups of 64-wide heads with the decay gradient would not fit a CU
  // (LDS is given out in steps of 1280 bytes).
  static constexpr int wc = p - C::kPad * (int)sizeof(T);
  // two buffers of gh, gl, wq and wk; then the decay gradient's partial sums
  static constexpr int kDecay = 4 * C::CH;
  static constexpr int red = 2 * kDecay;
  static constexpr int kSums = (4 + C::JW + C::NIB) * C::CH;  // two buffers of them too
  static constexpr int floats = red + (MODE >= kOutFwdDg ? 2 * kSums : 0);
  static constexpr int bytes = f + floats * 4;
};

// Element (r, c) of a tile of D columns in LDS.  bf16: a row starts 8 banks
// after the row before, and rows 8-15 of 16 swap the 16-byte chunks of each
// pair.  Then 16 rows read at one chunk, or at half a chunk, and, transposing,
// 8 rows of two chunks each meet every bank equally often, and every address
// is one lane offset plus a constant.  fp32: 4 banks further a row, for 16
// rows of one chunk and for rows e, 4 + e, 8 + e, 12 + e of four.
template <class T, int D>
__device__ __forceinline__ int at(int r, int c) {
  constexpr int EPV = Cfg<T>::EPV;
  if constexpr (Cfg<T>::kBf) return r * (D + Cfg<T>::kPad) + ((c / EPV) ^ ((r >> 3) & 1)) * EPV + c % EPV;
  return r * (D + Cfg<T>::kPad) + c;
}

// Element (i, j) of the scores (bf16: of each part's CH x CH), without padding
// (two workgroups a CU need the space): a row's 16-byte chunks are permuted
// instead.
template <class T>
__device__ __forceinline__ int at_p(int i, int j) {
  constexpr int EPV = Cfg<T>::EPV;
  return i * Cfg<T>::CH + ((j / EPV) ^ ((i >> 1) & 7)) * EPV + j % EPV;
}

// Barrier that orders LDS accesses only.  The fence of __syncthreads() also
// waits for every global access in flight, which here are the next chunk's
// loads and the previous one's stores.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A 64-bit value moved across lanes by a DPP control; lanes without a source
// (or outside the row mask) get 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double v) {
  const uint2 u = __builtin_bit_cast(uint2, v);
  const uint2 r{static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u.x), CTRL, ROWS, 0xF, true)),
                static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u.y), CTRL, ROWS, 0xF, true))};
  return __builtin_bit_cast(double, r);
}

// Inclusive sums over the lanes up to this one: inside rows of 16 lanes by
// shifts of 1, 2, 4, 8, then across rows by the broadcasts of lane 15 of each
// row to the next one and of lane 31 to the upper half.
__device__ __forceinline__ double prefix_sum(double v) {
  v += dpp_or_zero<0x111, 0xF>(v);
  v += dpp_or_zero<0x112, 0xF>(v);
  v += dpp_or_zero<0x114, 0xF>(v);
  v += dpp_or_zero<0x118, 0xF>(v);
  v += dpp_or_zero<0x142, 0xA>(v);
  v += dpp_or_zero<0x143, 0xC>(v);
  return v;
}

// A lane's 64-bit value, for all.
__device__ __forceinline__ double last_lane(double v, int lane) {
  const uint2 u = __builtin_bit_cast(uint2, v);
  const uint2 r{static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u.x), lane)),
                static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u.y), lane))};
  return __builtin_bit_cast(double, r);
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(
                 float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// Sums over the 16 lanes of a group (rotations by 8, 4, 2, 1), and over the
// four groups (swaps of rows and of halves); every lane gets the sum.
__device__ __forceinline__ float sum16(float v) {
  return dpp_add<0x121>(dpp_add<0x122>(dpp_add<0x124>(dpp_add<0x128>(v))));
}
__device__ __forceinline__ float sum_groups(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return ssm::xor_sum<32>(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

__device__ __forceinline__ f32x4_t mfma_bf16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

struct Pair64 { uint2 a, b; };
struct PairV4 { v4s a, b; };

// Four consecutive elements as floats, from LDS or global memory.
__device__ __forceinline__ f32x4_t load4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }
__device__ __forceinline__ f32x4_t load4(const bf16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return f32x4_t{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xffff0000u)};
}
// Two floats as bf16 (round to nearest, ties to even): one instruction.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}
__device__ __forceinline__ void store4(float* p, f32x4_t v) { *reinterpret_cast<f32x4_t*>(p) = v; }
__device__ __forceinline__ void store4(bf16_t* p, f32x4_t v) {
  *reinterpret_cast<uint2*>(p) = uint2{pack2(v[0], v[1]), pack2(v[2], v[3])};
}

__device__ __forceinline__ bf16x8_t load8(const bf16_t* p) { return *reinterpret_cast<const bf16x8_t*>(p); }
__device__ __forceinline__ bf16x8_t load44(const bf16_t* a, const bf16_t* b) {
  return __builtin_bit_cast(bf16x8_t,
                            (Pair64{*reinterpret_cast<const uint2*>(a), *reinterpret_cast<const uint2*>(b)}));
}
__device__ __forceinline__ bf16x8_t load8(const float*) { return bf16x8_t{}; }  // not reached

// Column c0 + l15 of rows t0 + 4 g .. + 3 and t0 + 16 + 4 g .. + 3 (t0 a
// multiple of 32): two transposing reads, in which lane s of a 16-lane group
// supplies the address of row s / 4, columns 4 (s % 4) .. + 3, and receives
// column s of the four rows.
template <int D>
__device__ __forceinline__ bf16x8_t read_tr(bf16_t* tile, int t0, int c0, int lane) {
  const int s = lane & 15, r = 4 * (lane >> 4) + (s >> 2), c = 4 * (s & 3);
  bf16_t* const p = tile + at<bf16_t, D>(r, c) + t0 * (D + Cfg<bf16_t>::kPad) + c0;
  const PairV4 v{__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p),
                 __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 16 * (D + Cfg<bf16_t>::kPad)))};
  return __builtin_bit_cast(bf16x8_t, v);
}

// nv rows of d elements, ld apart; accesses past the last one read zero and
// store nothing (offsets are range-checked in hardware, so no lane mask or
// branch splits the loads).  nv <= 0: an empty range (ld >= d there).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, int64_t ld, int nv, int d, int es) {
  const int bytes = ((nv - 1) * static_cast<int>(ld) + d) * es;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes > 0 ? bytes : 0, ssm::kBufWord3);
}

// Byte offset past any row range (which holds at most 64 x 2^24 bytes).
constexpr uint32_t kOutside = ssm::kBufOutside;

// A CH x D tile: global rows -> registers -> LDS.  Rows past the last token
// and channels past d are zero.
template <class T, int D>
struct Tile {
  using C = Cfg<T>;
  static constexpr int N = C::CH * D / C::EPV / kThreads;
  static constexpr int RPI = kThreads / (D / C::EPV);  // rows a load instruction covers
  u32x4_t r[N];
  uint32_t voff;  // the lane's byte offset in an instruction's rows
  int lds_off;
  __device__ __forceinline__ void init(int64_t ld, int d) {
    const int row = threadIdx.x / (D / C::EPV), col = threadIdx.x % (D / C::EPV) * C::EPV;
    voff = col < d ? static_cast<uint32_t>((row * ld + col) * sizeof(T)) : kOutside;
    lds_off = at<T, D>(row, col);
  }
  __device__ __forceinline__ void load(const T* p, int64_t ld, int nv, int d) {
    // one range per instruction (scalar work) keeps it to one lane offset
#pragma unroll
    for (int i = 0; i < N; i++)
      r[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                          rows_rsrc(p + i * RPI * ld, ld, nv - i * RPI, d, sizeof(T)), voff, 0, 0));
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int i = 0; i < N; i++) *reinterpret_cast<u32x4_t*>(lds + lds_off + at<T, D>(i * RPI, 0)) = r[i];
  }
};

// Four elements of a row range as loaded, and as floats.
template <class T> struct RawRows;
template <> struct RawRows<float> {
  typedef f32x4_t type;
  static __device__ __forceinline__ type load(__amdgpu_buffer_rsrc_t rs, uint32_t voff) {
    return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, voff, 0, 0));
  }
  static __device__ __forceinline__ f32x4_t f32(type v) { return v; }
};
template <> struct RawRows<bf16_t> {
  typedef uint2 type;
  static __device__ __forceinline__ type load(__amdgpu_buffer_rsrc_t rs, uint32_t voff) {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rs, voff, 0, 0));
  }
  static __device__ __forceinline__ f32x4_t f32(type u) {
    return f32x4_t{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                   __uint_as_float(u.y & 0xffff0000u)};
  }
};

__device__ __forceinline__ float widen(bf16x8_t v, int e) {
  const uint32_t u = __builtin_bit_cast(u32x4_t, v)[e / 2];
  return __uint_as_float(e % 2 ? u & 0xffff0000u : u << 16);
}

// Rounds the values to bf16; if more parts follow, leaves what the rounding
// lost.  In pairs: one conversion, and each half widened by a shift or a mask.
__device__ __forceinline__ bf16x8_t take_part(float (&v)[8], bool more) {
  u32x4_t p;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    p[i] = pack2(v[2 * i], v[2 * i + 1]);
    if (more) {
      v[2 * i] -= __uint_as_float(p[i] << 16);
      v[2 * i + 1] -= __uint_as_float(p[i] & 0xffff0000u);
    }
  }
  return __builtin_bit_cast(bf16x8_t, p);
}

__device__ __forceinline__ uint2 take_part(f32x4_t& v) {
  const uint2 p{pack2(v[0], v[1]), pack2(v[2], v[3])};
  v -= f32x4_t{__uint_as_float(p.x << 16), __uint_as_float(p.x & 0xffff0000u), __uint_as_float(p.y << 16),
               __uint_as_float(p.y & 0xffff0000u)};
  return p;
}

// Four output elements at a byte offset of a row range.
__device__ __forceinline__ void store_rows(__amdgpu_buffer_rsrc_t rs, uint32_t voff, f32x4_t v, float*) {
  __builtin_amdgcn_raw_buffer_store_b128(
      __builtin_bit_cast(__attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t, v), rs, voff, 0, 0);
}
__device__ __forceinline__ void store_rows(__amdgpu_buffer_rsrc_t rs, uint32_t voff, f32x4_t v, bf16_t*) {
  typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;
  __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])}, rs, voff, 0, 0);
}

// OT: type of the output rows, the io type or float.  PARTS: bf16 parts of
// the weighted V in the state's update, kParts where the state is an fp32
// output, kOutParts where it only reaches bf16 outputs.
template <class T, class OT, int DM, int DN, bool REV, int MODE, int PARTS>
__device__ __forceinline__ void run(const Args& a, const Run& r, uint32_t slot, int h, char* smem) {
  using C = Cfg<T>;
  using M = Lds<T, DM, DN, MODE>;
  constexpr bool kBf = C::kBf;
  constexpr int CH = C::CH, NIB = C::NIB, JW = C::JW;
  constexpr int MB = DM / 16, NB = DN / 64;
  constexpr bool kDg = MODE >= kOutFwdDg;
  constexpr int kStateParts = kDg ? kParts : kOutParts;
  constexpr int kDecayWave = REV ? 3 : 0;  // the wavefront with the fewest score blocks

  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int l15 = lane & 15, g = lane >> 4;

  Segment sg;
  const bool have = find_segment(a.sq, slot, CH, &sg);
  if (!have) return;
  if (MODE == kAgg && (REV ? sg.first : sg.last)) return;  // nothing after it

  T* const sQ = reinterpret_cast<T*>(smem + M::q);
  T* const sK = reinterpret_cast<T*>(smem + M::k);
  T* const sV = reinterpret_cast<T*>(smem + M::v);
  T* const sP = reinterpret_cast<T*>(smem + M::p);
  float* const sF = reinterpret_cast<float*>(smem + M::f);
  float* const sW = reinterpret_cast<float*>(smem + M::wc);
  const int n0 = wave * 16 * NB;  // this wavefront's state columns

  // the state entering the segment
  f32x4_t S[MB][NB];
  const bool split = r.seg != nullptr && !(sg.first && sg.last);
  const float* s_in = nullptr;
  if (MODE != kAgg) {
    if (split) s_in = r.seg + (static_cast<int64_t>(slot) * a.Hv + h) * a.dkdv;
    else if (r.s0) s_in = r.s0 + (static_cast<int64_t>(sg.seq) * a.Hv + h) * a.dkdv;
  }
  // a state in memory: element (m, n) at m sm + n sn
  auto state_rsrc = [&](const float* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p), 0, p ? a.dkdv * 4 : 0, ssm::kBufWord3);
  };
  auto state_off = [&](int mb, int nb) {
    const int m = 16 * mb + 4 * g, n = n0 + 16 * nb + l15;
    return m < r.dm && n < r.dn ? static_cast<uint32_t>(m * r.sm + n * r.sn) * 4u : kOutside;
  };
  {
    const __amdgpu_buffer_rsrc_t rs = state_rsrc(s_in);
#pragma unroll
    for (int mb = 0; mb < MB; mb++)
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          S[mb][nb][e] = __uint_as_float(
              __builtin_amdgcn_raw_buffer_load_b32(rs, state_off(mb, nb) + static_cast<uint32_t>(e * r.sm) * 4u, 0, 0));
  }

  const int len = sg.t1 - sg.t0;
  const int nch = (len + CH - 1) / CH;
  const T* const Qp = static_cast<const T*>(r.Q) + (h / r.gq) * r.dm;
  const T* const Kp = static_cast<const T*>(r.K) + (h / r.gk) * r.dm;
  const T* const Vp = static_cast<const T*>(r.V) + (h / r.gv) * r.dn;
  const T* const Xp = kDg ? static_cast<const T*>(r.X) + (h / r.gv) * r.dn : nullptr;

  Tile<T, DM> tq, tk;
  Tile<T, DN> tv;
  // rows of X, of this wavefront's row block, as operands of the scores
  constexpr int XF = MODE == kOutFwdDg ? DN * (int)sizeof(T) / 64 : 1;
  u32x4_t xf[XF];
  if constexpr (MODE != kAgg) tq.init(r.ldq, r.dm);
  tk.init(r.ldk, r.dm);
  tv.init(r.ldv, r.dn);
  constexpr int es_out = sizeof(OT);
  float g_next;  // this lane's log decay of the chunk being loaded
  // Loads of chunk c into registers; past the segment's end (the walk's last
  // step) the ranges are empty and nothing is fetched.
  auto chunk_rows = [&](int c, bool live) {
    const int nv = live ? sg.t1 - (sg.t0 + c * CH) : 0;
    return nv < CH ? nv : CH;
  };
  auto issue_decay = [&](int c, bool live) {
    const int64_t tb = sg.t0 + (live ? c * CH : 0);
    const int n = chunk_rows(c, live);
    const __amdgpu_buffer_rsrc_t rg = rows_rsrc(a.log_decay + tb * a.ld_decay + h, a.ld_decay, n, 1, 4);
    g_next = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
        rg, lane < n ? lane * static_cast<uint32_t>(a.ld_decay) * 4u : kOutside, 0, 0));
  };
  auto issue = [&](int c, bool live) {
    const int64_t tb = sg.t0 + (live ? c * CH : 0);
    const int n = chunk_rows(c, live);
    if constexpr (MODE != kAgg) tq.load(Qp + tb * r.ldq, r.ldq, n, r.dm);
    tk.load(Kp + tb * r.ldk, r.ldk, n, r.dm);
    tv.load(Vp + tb * r.ldv, r.ldv, n, r.dn);
  };
  auto issue_x = [&](int c, bool live) {
    if constexpr (MODE == kOutFwdDg) {
      const int row0 = 16 * (wave % NIB);
      const int64_t tb = sg.t0 + (live ? c * CH : 0) + row0;
      const __amdgpu_buffer_rsrc_t rx = rows_rsrc(Xp + tb * r.ldx, r.ldx, chunk_rows(c, live) - row0, r.dn, sizeof(T));
#pragma unroll
      for (int i = 0; i < XF; i++) {
        const int col = (4 * i + g) * C::EPV;
        xf[i] = __builtin_bit_cast(
            u32x4_t,
            __builtin_amdgcn_raw_buffer_load_b128(
                rx, col < r.dn ? static_cast<uint32_t>((l15 * r.ldx + col) * sizeof(T)) : kOutside, 0, 0));
      }
    }
  };
  // Sums of a chunk's log decays in 64 bits (base 2) and the weights made from them.
  auto decays = [&](int buf) {
    const double G = prefix_sum(decay_log2(g_next));
    const double tot = last_lane(G, CH - 1);
    if (lane < CH) {
      float* const o = sF + buf * M::kDecay;
      const float hi = static_cast<float>(G);
      o[lane] = hi;
      o[CH + lane] = static_cast<float>(G - static_cast<double>(hi));
      const float eg = exp2_split(G), er = exp2_split(tot - G);
      o[2 * CH + lane] = r.qs * (REV ? er : eg);
      o[3 * CH + lane] = r.ks * (REV ? eg : er);
    }
    if (lane == 0) sW[buf] = exp2_split(tot);
  };

  // Anchor states and their adjoints lie as the accumulators hold them.
  auto keep_state = [&](int c) {
    const int k = nch - 1 - c;
    if (k % kAnchor) return;
    const __amdgpu_buffer_rsrc_t ra =
        rows_rsrc(r.anchors + ((anchor_slot(sg, slot) + k / kAnchor) * a.Hv + h) * (DM * DN), 0, 1, DM * DN, 4);
#pragma unroll
    for (int mb = 0; mb < MB; mb++)
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, S[mb][nb]), ra, threadIdx.x * 16,
                                               (mb * NB + nb) * kThreads * 16, 0);
  };

  auto put = [&](int64_t tb, int nv, const f32x4_t (&Y)[NB][NIB]) {
    char* const o = static_cast<char*>(r.out) + (tb * r.ldo + h * r.dn) * es_out;
    const int n_out = r.out ? nv : 0;
#pragma unroll
    for (int b = 0; b < NIB; b++) {
      const __amdgpu_buffer_rsrc_t ro =
          rows_rsrc(o + 16 * b * r.ldo * es_out, r.ldo, n_out - 16 * b, r.dn, es_out);
#pragma unroll
      for (int nb = 0; nb < NB; nb++) {
        const int n = n0 + 16 * nb + 4 * g;
        store_rows(ro, n < r.dn ? static_cast<uint32_t>((l15 * r.ldo + n) * es_out) : kOutside, Y[nb][b],
                   static_cast<OT*>(nullptr));
      }
    }
  };

  // One lane per token: the decay gradient's sums inside chunk c, over i >= t
  // (forward run) or j <= t (reverse run).
  auto token_sums = [&](int c, int buf) {
    const float* const rint = sF + M::red + buf * M::kSums;
    double x = 0.0;
    if (lane < CH) {
#pragma unroll
      for (int w = 0; w < 4; w++) x += rint[w * CH + lane];
      if constexpr (MODE == kOutFwdDg) {
#pragma unroll
        for (int w = 0; w < JW; w++) x += rint[(4 + w) * CH + lane];
#pragma unroll
        for (int w = 0; w < NIB; w++) x -= rint[(4 + JW + w) * CH + lane];
      }
    }
    const double before = prefix_sum(x);
    if constexpr (MODE == kOutFwdDg) x += last_lane(before, CH - 1) - before;
    else x = before;
    const int t = sg.t0 + c * CH + lane;
    if (lane < CH && t < sg.t1) r.tok[static_cast<int64_t>(h) * a.sq.T + t] = static_cast<float>(x);
  };

  float decay_seg = 1.0f;
  if (nch > 0) {
    issue_decay(REV ? nch - 1 : 0, true);
    issue(REV ? nch - 1 : 0, true);
    issue_x(REV ? nch - 1 : 0, true);
    if (wave == kDecayWave) decays(0);
    // Global accesses retire in order: the loop waits for its loads by
    // counting what it issued after them.  Wait for the entering state and
    // issue as many (empty) stores here as a turn does, so that the first
    // turn counts like the others and no turn waits for its predecessor's
    // stores.
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    if constexpr (MODE != kAgg) {
      const __amdgpu_buffer_rsrc_t none = rows_rsrc(a.log_decay, 0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < NB * NIB; i++) store_rows(none, 16 * lane, f32x4_t{0.f, 0.f, 0.f, 0.f}, static_cast<OT*>(nullptr));
    }
  }
  for (int it = 0; it < nch; it++) {
    const int c = REV ? nch - 1 - it : it;
    const int64_t tb = sg.t0 + static_cast<int64_t>(c) * CH;
    const int nv = sg.t1 - static_cast<int>(tb) < CH ? sg.t1 - static_cast<int>(tb) : CH;
    const int buf = it & 1;
    int lane_now = lane;
    if constexpr (kDg) asm volatile("" : "+v"(lane_now));
    const int l15 = lane_now & 15, g = lane_now >> 4;
    const float* const gh = sF + buf * M::kDecay;
    const float* const gl = gh + CH;
    const float* const wq = gh + 2 * CH;
    const float* const wk = gh + 3 * CH;
    float* const sRint = sF + M::red + (kDg ? buf * M::kSums : 0);  // [4][CH]
    float* const sRow = sRint + 4 * CH;                            // [JW][CH]
    float* const sCol = sRow + JW * CH;                            // [NIB][CH]

    if (it > 0) lds_barrier();  // the previous chunk's readers are done
    if constexpr (MODE != kAgg) tq.store(sQ);
    tk.store(sK);
    tv.store(sV);
    lds_barrier();
    // what this chunk waits for comes before the next one's loads
    issue_decay(REV ? c - 1 : c + 1, it + 1 < nch);
    if constexpr (MODE == kAgg) issue(REV ? c - 1 : c + 1, it + 1 < nch);
    const float wc = sW[buf];

    f32x4_t Y[NB][NIB];
    if constexpr (MODE != kAgg) {
      // X where this wavefront's part of the output is
      typename RawRows<T>::type xv[kDg ? NB : 1][kDg ? NIB : 1];
      if constexpr (kDg) {
#pragma unroll
        for (int b = 0; b < NIB; b++) {
          const __amdgpu_buffer_rsrc_t rx = rows_rsrc(Xp + (tb + 16 * b) * r.ldx, r.ldx, nv - 16 * b, r.dn, sizeof(T));
#pragma unroll
          for (int nb = 0; nb < NB; nb++) {
            const int n = n0 + 16 * nb + 4 * g;
            xv[nb][b] = RawRows<T>::load(rx, n < r.dn ? static_cast<uint32_t>((l15 * r.ldx + n) * sizeof(T)) : kOutside);
          }
        }
      }
      // decayed scores of this wavefront's row block i, transposed: lane l
      // holds row i = l % 16 and four consecutive columns j
      const int ib = wave % NIB;
      const int i = 16 * ib + l15;
      const float ghi = gh[i], gli = gl[i];
      float rowsum = 0.0f;
      // the blocks that the mask leaves, and zeros in the other block of the
      // 32 columns that the product with V takes at once
      if constexpr (kBf) {
        if ((ib & 1) == (REV ? 1 : 0)) {
#pragma unroll
          for (int part = 0; part < kOutParts; part++)
            store4(sP + part * CH * CH + at_p<T>(i, 16 * (REV ? ib - 1 : ib + 1) + 4 * g), f32x4_t{0.f, 0.f, 0.f, 0.f});
        }
      }
      // operands of a block, read one block ahead
      constexpr int KF = DM * (int)sizeof(T) / 64, VF = MODE == kOutFwdDg ? DN * (int)sizeof(T) / 64 : 1;
      u32x4_t qf[KF], kf[KF], vf[VF];
      auto read_block = [&](int jb) {
        const T* const k0 = sK + at<T, DM>(l15, C::EPV * g) + 16 * jb * M::PM;
#pragma unroll
        for (int b = 0; b < KF; b++) kf[b] = *reinterpret_cast<const u32x4_t*>(k0 + 4 * C::EPV * b);
        if constexpr (MODE == kOutFwdDg) {
          const T* const v0 = sV + at<T, DN>(l15, C::EPV * g) + 16 * jb * M::PN;
#pragma unroll
          for (int b = 0; b < VF; b++) vf[b] = *reinterpret_cast<const u32x4_t*>(v0 + 4 * C::EPV * b);
        }
      };
      const T* const q0 = sQ + at<T, DM>(l15, C::EPV * g) + 16 * ib * M::PM;
#pragma unroll
      for (int b = 0; b < KF; b++) qf[b] = *reinterpret_cast<const u32x4_t*>(q0 + 4 * C::EPV * b);
      // blocks the mask leaves: up to ib, or from it (with JW > 1, each wavefront every JW-th)
      const int jb_end = REV ? NIB : ib + 1;
      int jb_first = wave / NIB;
      if (REV)
        while (jb_first < ib) jb_first += JW;
      if constexpr (MODE == kOutFwdDg) {
        for (int jb = jb_first; jb < NIB; jb += JW)
          if (jb >= jb_end && l15 < 4) sCol[ib * CH + 16 * jb + 4 * g + l15] = 0.0f;
      }
      if (jb_first < jb_end) read_block(jb_first);
#pragma unroll 1
      for (int jb = jb_first; jb < jb_end; jb += JW) {
        {
          f32x4_t p;
          float colsum[4];
          f32x4_t acc{0.f, 0.f, 0.f, 0.f};
          f32x4_t acx{0.f, 0.f, 0.f, 0.f};
          if constexpr (kBf) {
#pragma unroll
            for (int b = 0; b < KF; b++)
              acc = mfma_bf16(__builtin_bit_cast(bf16x8_t, kf[b]), __builtin_bit_cast(bf16x8_t, qf[b]), acc);
            if constexpr (MODE == kOutFwdDg) {
              // the other pair's scores, X_i . V_j
#pragma unroll
              for (int b = 0; b < VF; b++)
                acx = mfma_bf16(__builtin_bit_cast(bf16x8_t, vf[b]), __builtin_bit_cast(bf16x8_t, xf[b]), acx);
            }
          } else {
#pragma unroll
            for (int b = 0; b < KF; b++) {
              const f32x4_t ka = __builtin_bit_cast(f32x4_t, kf[b]), qa = __builtin_bit_cast(f32x4_t, qf[b]);
#pragma unroll
              for (int e = 0; e < 4; e++) acc = mfma_f32(ka[e], qa[e], acc);
            }
            if constexpr (MODE == kOutFwdDg) {
#pragma unroll
              for (int b = 0; b < VF; b++) {
                const f32x4_t va = __builtin_bit_cast(f32x4_t, vf[b]), xa = __builtin_bit_cast(f32x4_t, xf[b]);
#pragma unroll
                for (int e = 0; e < 4; e++) acx = mfma_f32(va[e], xa[e], acx);
              }
            }
          }
          if (jb + JW < jb_end) read_block(jb + JW);
          const int j0 = 16 * jb + 4 * g;
          const f32x4_t ghj = load4(gh + j0), glj = load4(gl + j0);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int j = j0 + e;
            const float d = REV ? (ghj[e] - ghi) + (glj[e] - gli) : (ghi - ghj[e]) + (gli - glj[e]);
            const bool in = REV ? j >= i : j <= i;
            p[e] = in ? acc[e] * (ssm::fast_exp2(d) * (r.qs * r.ks)) : 0.0f;
            if constexpr (MODE == kOutFwdDg) {
              const float m = j < i ? p[e] * acx[e] : 0.0f;
              rowsum += m;
              colsum[e] = m;
            }
          }
          if constexpr (kBf) {
#pragma unroll
            for (int part = 0; part < kOutParts; part++)
              *reinterpret_cast<uint2*>(sP + part * CH * CH + at_p<T>(i, 16 * jb + 4 * g)) = take_part(p);
          } else {
            store4(sP + at_p<T>(i, 16 * jb + 4 * g), p);
          }
          if constexpr (MODE == kOutFwdDg) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float t = sum16(colsum[e]);
              s = l15 == e ? t : s;
            }
            if (l15 < 4) sCol[ib * CH + 16 * jb + 4 * g + l15] = s;
          }
        }
      }
      if constexpr (MODE == kOutFwdDg) {
        rowsum = sum_groups(rowsum);
        if (g == 0) sRow[(wave / NIB) * CH + i] = rowsum;
      }

      if constexpr (kDg) keep_state(c);
      // the next chunk's loads: after the scores, whose registers they take
      // (with the decay gradient's operands, after the state's part, which
      // takes more, and in fp32 after the product with V: 65536 bf16 tokens,
      // 16 heads of 128 take 1.47 ms, 1.50 after that product; 32768 fp32
      // tokens 1.72 ms, 1.70 after it)
      if constexpr (!kDg) issue(REV ? c - 1 : c + 1, it + 1 < nch);

      // the state's part, transposed: rows n of this wavefront, columns i
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
#pragma unroll
        for (int b = 0; b < NIB; b++) Y[nb][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if constexpr (kBf) {
#pragma unroll
        for (int kb = 0; kb < MB / 2; kb++) {
          bf16x8_t qf[NIB];
#pragma unroll
          for (int b = 0; b < NIB; b++) {
            const int q = at<T, DM>(16 * b + l15, 4 * g) + 32 * kb;
            qf[b] = load44(sQ + q, sQ + q + 16);
          }
#pragma unroll
          for (int nb = 0; nb < NB; nb++) {
            float s[8];
#pragma unroll
            for (int e = 0; e < 8; e++) s[e] = S[2 * kb + e / 4][nb][e % 4];
#pragma unroll
            for (int part = 0; part < kStateParts; part++) {
              const bf16x8_t sf = take_part(s, part + 1 < kStateParts);
#pragma unroll
              for (int b = 0; b < NIB; b++) Y[nb][b] = mfma_bf16(sf, qf[b], Y[nb][b]);
            }
          }
        }
      } else {
#pragma unroll
        for (int mb = 0; mb < MB; mb++)
#pragma unroll
          for (int b = 0; b < NIB; b++) {
            const f32x4_t q = load4(sQ + at<T, DM>(16 * b + l15, 16 * mb + 4 * g));
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
              for (int e = 0; e < 4; e++) Y[nb][b] = mfma_f32(S[mb][nb][e], q[e], Y[nb][b]);
          }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < NIB; b++) {
        const float w = wq[16 * b + l15];
        float dot = 0.0f;
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
          Y[nb][b] = Y[nb][b] * w;
          if constexpr (kDg) {
            const f32x4_t x = RawRows<T>::f32(xv[nb][b]);
#pragma unroll
            for (int e = 0; e < 4; e++) dot = fmaf(x[e], Y[nb][b][e], dot);
          }
        }
        if constexpr (kDg) {
          dot = sum_groups(dot);
          if (g == 0) sRint[wave * CH + 16 * b + l15] = dot;
        }
      }
    }
    // while the other wavefronts have scores left
    if (wave == kDecayWave) {
      if (it + 1 < nch) decays(buf ^ 1);
      if constexpr (kDg)
        if (it > 0) token_sums(REV ? c + 1 : c - 1, buf ^ 1);
    }
    if constexpr (MODE != kAgg) lds_barrier();  // scores and partial sums are in LDS

    if constexpr (kDg && kBf) {
      issue(REV ? c - 1 : c + 1, it + 1 < nch);
      issue_x(REV ? c - 1 : c + 1, it + 1 < nch);
    } else {
      __builtin_amdgcn_sched_barrier(0);
    }
    // V of this wavefront's columns, tokens along the lane's elements
    if constexpr (kBf) {
      bf16x8_t vf[CH / 32][NB];
#pragma unroll
      for (int kb = 0; kb < CH / 32; kb++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
          vf[kb][nb] = read_tr<DN>(sV, 32 * kb, n0 + 16 * nb, lane_now);
        }
      if constexpr (MODE != kAgg) {
#pragma unroll
        for (int b = 0; b < NIB; b++)
#pragma unroll
          for (int kb = 0; kb < CH / 32; kb++)
            if (REV ? 2 * kb + 1 >= b : 2 * kb <= b) {
#pragma unroll
              for (int part = 0; part < kOutParts; part++) {
                const T* const sp = sP + part * CH * CH;
                const bf16x8_t pf = load44(sp + at_p<T>(16 * b + l15, 32 * kb + 4 * g),
                                           sp + at_p<T>(16 * b + l15, 32 * kb + 16 + 4 * g));
#pragma unroll
                for (int nb = 0; nb < NB; nb++) Y[nb][b] = mfma_bf16(vf[kb][nb], pf, Y[nb][b]);
              }
            }
        put(tb, nv, Y);
      }
      __builtin_amdgcn_sched_barrier(0);
      // the state's update
#pragma unroll
      for (int mb = 0; mb < MB; mb++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) S[mb][nb] = S[mb][nb] * wc;
#pragma unroll
      for (int kb = 0; kb < CH / 32; kb++) {
        const f32x4_t w0 = load4(wk + 32 * kb + 4 * g), w1 = load4(wk + 32 * kb + 16 + 4 * g);
        bf16x8_t vw[NB][PARTS];
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
          float u[8];
#pragma unroll
          for (int e = 0; e < 8; e++) u[e] = widen(vf[kb][nb], e) * (e < 4 ? w0[e % 4] : w1[e % 4]);
#pragma unroll
          for (int part = 0; part < PARTS; part++) vw[nb][part] = take_part(u, part + 1 < PARTS);
        }
#pragma unroll
        for (int mb = 0; mb < MB; mb++) {
          const bf16x8_t kf = read_tr<DM>(sK, 32 * kb, 16 * mb, lane_now);
#pragma unroll
          for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int part = 0; part < PARTS; part++) S[mb][nb] = mfma_bf16(kf, vw[nb][part], S[mb][nb]);
        }
      }
    } else {
#pragma unroll
      for (int mb = 0; mb < MB; mb++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) S[mb][nb] = S[mb][nb] * wc;
#pragma unroll
      for (int tk16 = 0; tk16 < NIB; tk16++) {
        float vf[4][NB];
#pragma unroll
        for (int e = 0; e < 4; e++)
#pragma unroll
          for (int nb = 0; nb < NB; nb++)
            vf[e][nb] = sV[at<T, DN>(16 * tk16 + 4 * g + e, n0 + 16 * nb + l15)];
        if constexpr (MODE != kAgg) {
#pragma unroll
          for (int b = 0; b < NIB; b++)
            if (REV ? tk16 >= b : tk16 <= b) {
              const f32x4_t p = load4(sP + at_p<T>(16 * b + l15, 16 * tk16 + 4 * g));
#pragma unroll
              for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int e = 0; e < 4; e++) Y[nb][b] = mfma_f32(vf[e][nb], p[e], Y[nb][b]);
            }
        }
        const f32x4_t w = load4(wk + 16 * tk16 + 4 * g);
#pragma unroll
        for (int mb = 0; mb < MB; mb++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float kf = sK[at<T, DM>(16 * tk16 + 4 * g + e, 16 * mb + l15)];
#pragma unroll
            for (int nb = 0; nb < NB; nb++) S[mb][nb] = mfma_f32(kf, vf[e][nb] * w[e], S[mb][nb]);
          }
      }
      if constexpr (kDg) {
        issue(REV ? c - 1 : c + 1, it + 1 < nch);
        issue_x(REV ? c - 1 : c + 1, it + 1 < nch);
      }
      if constexpr (MODE != kAgg) put(tb, nv, Y);
    }
    if constexpr (MODE == kAgg) decay_seg *= wc;

  }
  if constexpr (kDg) {
    if (nch > 0) {
      lds_barrier();
      if (wave == kDecayWave) token_sums(REV ? 0 : nch - 1, (nch - 1) & 1);
    }
  }

  // the state leaving the segment: the aggregate, or the sequence's
  float* s_out = nullptr;
  if (MODE == kAgg) {
    s_out = r.seg + (static_cast<int64_t>(slot) * a.Hv + h) * a.dkdv;
    if (threadIdx.x == 0) r.seg_decay[static_cast<int64_t>(slot) * a.Hv + h] = decay_seg;
  } else if (r.s_end && (REV ? sg.first : sg.last)) {
    s_out = r.s_end + (static_cast<int64_t>(sg.seq) * a.Hv + h) * a.dkdv;
  }
  if (s_out) {
    const __amdgpu_buffer_rsrc_t rs = state_rsrc(s_out);
#pragma unroll
    for (int mb = 0; mb < MB; mb++)
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[mb][nb][e]), rs,
                                                state_off(mb, nb) + static_cast<uint32_t>(e * r.sm) * 4u, 0, 0);
  }
}

// The workgroup's segment, head and run.  Workgroups go round-robin over the
// 8 XCDs: the runs of one head, which read the same rows, follow one another
// on one XCD and find the rows in its L2.
struct Work {
  uint32_t slot;
  int h, z;
  bool any;
};

__device__ __forceinline__ Work work_of(const Args& a) {
  const uint32_t nz = static_cast<uint32_t>(a.nz);
  const uint32_t i = blockIdx.x / 8, u = i / nz * 8 + blockIdx.x % 8;
  Work w;
  w.any = u < a.units;
  w.slot = u / static_cast<uint32_t>(a.Hv);
  w.h = static_cast<int>(u % static_cast<uint32_t>(a.Hv));
  w.z = a.run_of[i % nz];
  return w;
}

// Workgroups that share a CU: as many as the state's registers leave room
// for (the LDS does too).
constexpr int wgs_per_cu(int dk, int dv, int kind) {
  const int n = dk * dv > 64 * 64 ? 2 : 3;
  return kind == kAggregate || kind == kAggregateOut ? n + 1 : n;
}

// Kinds: kGrad... with PT the type of dq and dk, float where the value heads
// of a key head are summed afterwards.
template <class T, class PT, int DK, int DV, int KIND>
__global__ __launch_bounds__(kThreads, wgs_per_cu(DK, DV, KIND)) void k_linattn(Args a) {
  extern __shared__ __attribute__((aligned(16))) char smem_la[];
  const Work w = work_of(a);
  if (!w.any) return;
  if constexpr (KIND == kForward) {
    run<T, T, DK, DV, false, kOut, kOutParts>(a, a.run[0], w.slot, w.h, smem_la);
  } else if constexpr (KIND == kForwardState) {
    run<T, T, DK, DV, false, kOut, kParts>(a, a.run[0], w.slot, w.h, smem_la);
  } else if constexpr (KIND == kAggregate || KIND == kAggregateOut) {
    constexpr int P = KIND == kAggregate ? kParts : kOutParts;
    if (w.z == 0) run<T, T, DK, DV, false, kAgg, P>(a, a.run[0], w.slot, w.h, smem_la);
    else run<T, T, DK, DV, true, kAgg, P>(a, a.run[1], w.slot, w.h, smem_la);
  } else {
    constexpr bool dg = KIND == kGradDecay;
    if (w.z == 0) run<T, PT, DV, DK, false, dg ? kOutFwdDg : kOut, dg ? kParts : kOutParts>(a, a.run[0], w.slot, w.h, smem_la);
    else if (w.z == 1) run<T, PT, DV, DK, true, dg ? kOutRevDg : kOut, kParts>(a, a.run[1], w.slot, w.h, smem_la);
    else run<T, T, DK, DV, true, kOut, kOutParts>(a, a.run[2], w.slot, w.h, smem_la);
  }
}

constexpr int max2(int a, int b) { return a > b ? a : b; }

template <class T, int DK, int DV, int KIND>
constexpr int lds_bytes() {
  if (KIND == kForward || KIND == kForwardState) return Lds<T, DK, DV, kOut>::bytes;
  if (KIND == kAggregate || KIND == kAggregateOut) return Lds<T, DK, DV, kAgg>::bytes;
  if (KIND == kGradDecay) return max2(Lds<T, DV, DK, kOutFwdDg>::bytes, Lds<T, DK, DV, kOut>::bytes);
  return max2(Lds<T, DV, DK, kOut>::bytes, Lds<T, DK, DV, kOut>::bytes);
}

template <class T, class PT, int DK, int DV, int KIND>
hipError_t launch_one(const Args& a, hipStream_t st) {
  constexpr int lds = lds_bytes<T, DK, DV, KIND>();
  static_assert(lds <= 80 * 1024, "two workgroups share a CU's 160 KB");
  auto kern = k_linattn<T, PT, DK, DV, KIND>;
  if constexpr (lds > 64 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const uint32_t grid = (a.units + 7) / 8 * 8 * static_cast<uint32_t>(a.nz);
  kern<<<grid, kThreads, lds, st>>>(a);
  return hipGetLastError();
}

template <class T, int DK, int DV>
hipError_t launch_kind(Kernel k, const Args& a, hipStream_t st) {
  if (k == kForward) return launch_one<T, T, DK, DV, kForward>(a, st);
  if (k == kForwardState) return launch_one<T, T, DK, DV, kForwardState>(a, st);
  if constexpr (Cfg<T>::kBf) {  // fp32 has no parts
    if (k == kAggregateOut) return launch_one<T, T, DK, DV, kAggregateOut>(a, st);
  }
  if (k == kAggregate || k == kAggregateOut) return launch_one<T, T, DK, DV, kAggregate>(a, st);
  if (a.sum_heads)
    return k == kGradDecay ? launch_one<T, float, DK, DV, kGradDecay>(a, st)
                           : launch_one<T, float, DK, DV, kGradPlain>(a, st);
  return k == kGradDecay ? launch_one<T, T, DK, DV, kGradDecay>(a, st) : launch_one<T, T, DK, DV, kGradPlain>(a, st);
}

}  // namespace

}  // namespace la
