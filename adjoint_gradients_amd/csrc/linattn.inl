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
// forward run stores the states entering each chunk so that the reverse run
// can form <S, D>.
//
// One workgroup of four wavefronts walks the chunks of one segment of one
// sequence for one head.  The state stays in the accumulators of v_mfma
// 16x16 tiles, each wavefront holding all dm rows of its quarter of the dn
// columns; as laid out there it is itself the operand of Q S, with the rows
// of Q read in the matching order, so it never passes through LDS.  Q, K, V
// go through LDS; the next chunk's tiles are loaded into registers while the
// current one is computed.
//
// Rounding: products are bf16 x bf16 summed in fp32 (or fp32 throughout).
// The decayed scores are rounded to bf16 before they multiply V, and the
// state to bf16 where it multiplies Q: both errors are of the size of the
// output's own rounding.  What ends in an fp32 output (states, decay
// gradient) is split into bf16 parts that together hold the fp32 value to
// 2^-17: the weighted V of the state's update, and the state in the runs
// that form the decay gradient.
#include "linattn.hpp"
#include "ssm_common.hpp"

namespace la {

namespace {

using ssm::bf16_t;
using ssm::bf16x8_t;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kThreads = 256;  // four wavefronts
constexpr float kLn2 = 0.69314718055994531f;

// Modes of a run.
constexpr int kOut = 0;       // out
constexpr int kAgg = 1;       // only the state's sum over the segment
constexpr int kOutFwdDg = 2;  // out, the decay gradient's forward terms, the chunk states
constexpr int kOutRevDg = 3;  // out and the decay gradient

template <class T>
struct Cfg {
  static constexpr bool kBf = sizeof(T) == 2;
  static constexpr int CH = chunk_tokens(kBf);
  static constexpr int NIB = CH / 16;      // 16-token blocks
  static constexpr int JW = 4 / NIB;       // wavefronts sharing a row block of the scores
  static constexpr int EPV = 16 / sizeof(T);
};

// LDS of a run, in bytes.
template <class T, int DM, int DN, int MODE>
struct Lds {
  using C = Cfg<T>;
  static constexpr int PM = DM + C::EPV, PN = DN + C::EPV;
  static constexpr int q = 0;
  static constexpr int k = q + (MODE == kAgg ? 0 : C::CH * PM * (int)sizeof(T));
  static constexpr int v = k + C::CH * PM * (int)sizeof(T);
  static constexpr int x = v + C::CH * PN * (int)sizeof(T);
  static constexpr int p = x + (MODE == kOutFwdDg ? C::CH * PN * (int)sizeof(T) : 0);
  static constexpr int f = p + (MODE == kAgg ? 0 : C::CH * C::CH * (int)sizeof(T));
  // gh, gl, wq; two buffers of wk and of wc; then the decay gradient's partial sums
  static constexpr int wk = 3 * C::CH;
  static constexpr int wc = wk + 2 * C::CH;
  static constexpr int red = wc + 4;
  static constexpr int floats = red + (MODE >= kOutFwdDg ? (4 + C::JW + C::NIB) * C::CH + 4 : 0);
  static constexpr int bytes = f + floats * 4;
};

// Element (r, c) of a tile of D columns in LDS.  Rows start 16 bytes later in
// the banks than the row before: 16 rows read at one chunk of 16 bytes, or at
// half a chunk, meet every bank equally often, and every address is one lane
// offset plus a constant.  (The transposing reads meet half the banks twice;
// a permutation of the chunks avoids that but needs an address of its own
// for most reads, about a hundred registers.)
template <class T, int D>
__device__ __forceinline__ int at(int r, int c) { return r * (D + Cfg<T>::EPV) + c; }

// Element (i, j) of the scores, without padding (two workgroups a CU need the
// space): a row's 16-byte chunks are permuted instead.
template <class T>
__device__ __forceinline__ int at_p(int i, int j) {
  constexpr int EPV = Cfg<T>::EPV;
  return i * Cfg<T>::CH + ((j / EPV) ^ ((i >> 1) & 7)) * EPV + j % EPV;
}

struct Segment {
  int32_t seq;
  int32_t t0, t1;      // its tokens
  int32_t chunk_slot;  // of its first chunk
  bool first, last;    // of its sequence
};

// The segment of a slot; false if the slot has none.  The sequence is found
// by bisection over the first slots start[s] / L + s, which increase with s.
__device__ __forceinline__ bool find_segment(const Seqs& sq, uint32_t slot, int ch, Segment* o) {
  const uint32_t L = static_cast<uint32_t>(sq.L), T = static_cast<uint32_t>(sq.T);
  const uint32_t n = T / static_cast<uint32_t>(sq.S);
  auto start = [&](int32_t s) -> uint32_t {
    if (!sq.start) return n * static_cast<uint32_t>(s);
    const int32_t v = sq.start[s];
    return v < 0 ? 0u : static_cast<uint32_t>(v) > T ? T : static_cast<uint32_t>(v);
  };
  int32_t lo = 0, hi = sq.S - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) / 2;
    if (start(mid) / L + static_cast<uint32_t>(mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const uint32_t a = start(lo);
  uint32_t b = start(lo + 1);
  b = b < a ? a : b;
  const uint32_t base = a / L + static_cast<uint32_t>(lo);
  if (slot < base) return false;
  const uint32_t j = slot - base;
  const uint32_t nseg = (b - a + L - 1) / L;
  if (j >= (nseg ? nseg : 1u)) return false;
  o->seq = lo;
  o->t0 = static_cast<int32_t>(a + j * L);
  o->t1 = static_cast<int32_t>(b - a - j * L < L ? b : a + (j + 1) * L);
  o->chunk_slot = static_cast<int32_t>(a / static_cast<uint32_t>(ch)) + lo + static_cast<int32_t>(j * (L / ch));
  o->first = j == 0;
  o->last = j + 1 >= nseg;
  return true;
}

// Barrier that orders LDS accesses only.  The fence of __syncthreads() also
// waits for every global access in flight, which here are the next chunk's
// loads and the previous one's stores.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 2^x of a 64-bit x, to fp32 accuracy also for large |x|.
__device__ __forceinline__ float exp2_split(double x) {
  const float h = static_cast<float>(x);
  const float l = static_cast<float>(x - static_cast<double>(h));
  const float e = ssm::fast_exp2(h);
  return fmaf(e, l * kLn2, e);
}

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

template <int D>
__device__ __forceinline__ float xor_add(float v) { return v + __shfl_xor(v, D, 64); }

// Sums over the 16 lanes of a group, and over the four groups.
__device__ __forceinline__ float sum16(float v) { return xor_add<8>(xor_add<4>(xor_add<2>(xor_add<1>(v)))); }
__device__ __forceinline__ float sum_groups(float v) { return xor_add<32>(xor_add<16>(v)); }

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
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return static_cast<uint32_t>(ssm::f32_to_bf16(a)) | (static_cast<uint32_t>(ssm::f32_to_bf16(b)) << 16);
}
__device__ __forceinline__ void store4(float* p, f32x4_t v) { *reinterpret_cast<f32x4_t*>(p) = v; }
__device__ __forceinline__ void store4(bf16_t* p, f32x4_t v) {
  *reinterpret_cast<uint2*>(p) = uint2{pack2(v[0], v[1]), pack2(v[2], v[3])};
}

__device__ __forceinline__ bf16x8_t load8(const bf16_t* p) { return *reinterpret_cast<const bf16x8_t*>(p); }
__device__ __forceinline__ bf16x8_t load8(const float*) { return bf16x8_t{}; }  // not reached

// Rows t0 .. t0 + 7 (t0 a multiple of 8, one per 16-lane group) of column
// c0 + l15: two transposing reads, in which lane s of a group supplies the
// address of row s / 4, columns 4 (s % 4) .. + 3, and receives column s of
// the four rows.
template <int D>
__device__ __forceinline__ bf16x8_t read_tr(bf16_t* tile, int t0, int c0, int l15) {
  const int r = t0 + (l15 >> 2), c = c0 + 4 * (l15 & 3);
  const PairV4 p{__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(tile + at<bf16_t, D>(r, c))),
                 __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(tile + at<bf16_t, D>(r + 4, c)))};
  return __builtin_bit_cast(bf16x8_t, p);
}

// Rows of d elements, ld apart, from a chunk's first token on; accesses past
// row nv read zero and store nothing (offsets are range-checked in hardware,
// so no lane mask or branch splits the loads).  A null base is an empty range.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, int64_t ld, int nv, int d, int es) {
  const int bytes = p && nv > 0 ? static_cast<int>(((nv - 1) * ld + d) * es) : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, ssm::kBufWord3);
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
  typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4;
  u32x4 r[N];
  uint32_t voff, step;  // the lane's byte offset; bytes between the rows of successive instructions
  int lds_off;
  __device__ __forceinline__ void init(int64_t ld, int d) {
    const int row = threadIdx.x / (D / C::EPV), col = threadIdx.x % (D / C::EPV) * C::EPV;
    voff = col < d ? static_cast<uint32_t>((row * ld + col) * sizeof(T)) : kOutside;
    step = static_cast<uint32_t>(RPI * ld * sizeof(T));
    lds_off = at<T, D>(row, col);
  }
  __device__ __forceinline__ void load(const T* p, int64_t ld, int nv, int d) {
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(p, ld, nv, d, sizeof(T));
#pragma unroll
    for (int i = 0; i < N; i++) {
      // a lane past d stays outside: steps stay under 2^30 bytes in all
      r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, voff + i * step, 0, 0));
    }
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int i = 0; i < N; i++) *reinterpret_cast<u32x4*>(lds + lds_off + at<T, D>(i * RPI, 0)) = r[i];
  }
};

// Four output elements at a byte offset of a row range.
__device__ __forceinline__ void store_rows(__amdgpu_buffer_rsrc_t rs, uint32_t voff, f32x4_t v, float*) {
  __builtin_amdgcn_raw_buffer_store_b128(
      __builtin_bit_cast(__attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t, v), rs, voff, 0, 0);
}
__device__ __forceinline__ void store_rows(__amdgpu_buffer_rsrc_t rs, uint32_t voff, f32x4_t v, bf16_t*) {
  typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2;
  __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])}, rs, voff, 0, 0);
}
__device__ __forceinline__ f32x4_t load_rows(__amdgpu_buffer_rsrc_t rs, uint32_t voff, const float*) {
  return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, voff, 0, 0));
}
__device__ __forceinline__ f32x4_t load_rows(__amdgpu_buffer_rsrc_t rs, uint32_t voff, const bf16_t*) {
  const auto u = __builtin_amdgcn_raw_buffer_load_b64(rs, voff, 0, 0);
  return f32x4_t{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u), __uint_as_float(u[1] << 16),
                 __uint_as_float(u[1] & 0xffff0000u)};
}

// OT: type of the output rows, the io type or float.
template <class T, class OT, int DM, int DN, bool REV, int MODE>
__device__ __forceinline__ void run(const Args& a, const Run& r, char* smem) {
  using C = Cfg<T>;
  using M = Lds<T, DM, DN, MODE>;
  constexpr bool kBf = C::kBf;
  constexpr int CH = C::CH, NIB = C::NIB, JW = C::JW;
  constexpr int MB = DM / 16, NB = DN / 64;
  constexpr bool kDg = MODE >= kOutFwdDg;
  constexpr int kDecayWave = REV ? 3 : 0;  // the wavefront with the fewest score blocks

  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int l15 = lane & 15, g = lane >> 4;
  const int h = blockIdx.y;
  const uint32_t slot = blockIdx.x;

  if (!r.K) return;  // a run that this launch leaves out
  Segment sg;
  const bool have = find_segment(a.sq, slot, CH, &sg);
  if constexpr (MODE == kOutRevDg) {
    if (r.dg_seg && !have && threadIdx.x == 0) r.dg_seg[static_cast<int64_t>(slot) * a.Hv + h] = 0.0;
  }
  if (!have) return;
  if (MODE == kAgg && (REV ? sg.first : sg.last)) return;  // nothing after it

  T* const sQ = reinterpret_cast<T*>(smem + M::q);
  T* const sK = reinterpret_cast<T*>(smem + M::k);
  T* const sV = reinterpret_cast<T*>(smem + M::v);
  T* const sX = reinterpret_cast<T*>(smem + M::x);
  T* const sP = reinterpret_cast<T*>(smem + M::p);
  float* const sF = reinterpret_cast<float*>(smem + M::f);
  float* const sRint = sF + M::red;        // [4][CH]
  float* const sRow = sRint + 4 * CH;      // [JW][CH]
  float* const sCol = sRow + JW * CH;      // [NIB][CH]
  float* const sDot = sCol + NIB * CH;     // [4]

  const int n0 = wave * 16 * NB;  // this wavefront's state columns

  // the state entering the segment
  f32x4_t S[MB][NB];
  const bool split = r.seg != nullptr && !(sg.first && sg.last);
  const float* s_in = nullptr;
  if (MODE != kAgg) {
    if (split) s_in = r.seg + (static_cast<int64_t>(slot) * a.Hv + h) * a.dkdv;
    else if (r.s0) s_in = r.s0 + (static_cast<int64_t>(sg.seq) * a.Hv + h) * a.dkdv;
  }
#pragma unroll
  for (int mb = 0; mb < MB; mb++)
#pragma unroll
    for (int nb = 0; nb < NB; nb++) {
      const int m = 16 * mb + 4 * g, n = n0 + 16 * nb + l15;
      S[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (s_in && m < r.dm && n < r.dn)
#pragma unroll
        for (int e = 0; e < 4; e++) S[mb][nb][e] = s_in[(m + e) * r.sm + n * r.sn];
    }

  const int len = sg.t1 - sg.t0;
  const int nch = (len + CH - 1) / CH;
  const T* const Qp = static_cast<const T*>(r.Q) + (h / r.gq) * r.dm;
  const T* const Kp = static_cast<const T*>(r.K) + (h / r.gk) * r.dm;
  const T* const Vp = static_cast<const T*>(r.V) + (h / r.gv) * r.dn;
  const T* const Xp = kDg ? static_cast<const T*>(r.X) + (h / r.gv) * r.dn : nullptr;

  Tile<T, DM> tq, tk;
  Tile<T, DN> tv, tx;
  if constexpr (MODE != kAgg) tq.init(r.ldq, r.dm);
  tk.init(r.ldk, r.dm);
  tv.init(r.ldv, r.dn);
  if constexpr (MODE == kOutFwdDg) tx.init(r.ldx, r.dn);
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
    if constexpr (MODE == kOutFwdDg) tx.load(Xp + tb * r.ldx, r.ldx, n, r.dn);
  };
  // Sums of a chunk's log decays in 64 bits (base 2) and the weights made
  // from them.  A decay below e^-13000 is taken as that: both are zero in
  // every product, and -inf would make a NaN of inf - inf.
  auto decays = [&](int buf) {
    const double G =
        prefix_sum(static_cast<double>(g_next < -13000.0f ? -13000.0f : g_next) * 1.4426950408889634);
    const uint2 gb = __builtin_bit_cast(uint2, G);
    const uint2 tb{static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(gb.x), CH - 1)),
                   static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(gb.y), CH - 1))};
    const double tot = __builtin_bit_cast(double, tb);
    if (lane < CH) {
      const float hi = static_cast<float>(G);
      sF[lane] = hi;
      sF[CH + lane] = static_cast<float>(G - static_cast<double>(hi));
      const float eg = exp2_split(G), er = exp2_split(tot - G);
      sF[2 * CH + lane] = r.qs * (REV ? er : eg);
      sF[M::wk + buf * CH + lane] = r.ks * (REV ? eg : er);
    }
    if (lane == 0) sF[M::wc + buf] = exp2_split(tot);
  };

  auto chunk_state = [&](int c) {
    return reinterpret_cast<f32x4_t*>(r.chunk_states +
                                      (static_cast<int64_t>(sg.chunk_slot + c) * a.Hv + h) * (DM * DN));
  };

  float decay_seg = 1.0f;
  double dg_sum = 0.0;
  if (nch > 0) {
    issue_decay(REV ? nch - 1 : 0, true);
    issue(REV ? nch - 1 : 0, true);
    if (wave == kDecayWave) decays(0);
    // Global accesses retire in order: the loop waits for its loads by
    // counting what it issued after them.  Wait for the entering state and
    // issue as many (empty) stores here as a turn does, so that the first
    // turn counts like the others and no turn waits for its predecessor's
    // stores.
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    if constexpr (MODE != kAgg) {
      const __amdgpu_buffer_rsrc_t none = rows_rsrc(nullptr, 0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < NB * NIB; i++) store_rows(none, 16 * lane, f32x4_t{0.f, 0.f, 0.f, 0.f}, static_cast<OT*>(nullptr));
      if constexpr (MODE == kOutFwdDg)
#pragma unroll
        for (int i = 0; i < MB * NB; i++) store_rows(none, 16 * lane, f32x4_t{0.f, 0.f, 0.f, 0.f}, static_cast<float*>(nullptr));
    }
  }
  for (int it = 0; it < nch; it++) {
    const int c = REV ? nch - 1 - it : it;
    const int64_t tb = sg.t0 + static_cast<int64_t>(c) * CH;
    const int nv = sg.t1 - static_cast<int>(tb) < CH ? sg.t1 - static_cast<int>(tb) : CH;
    const int buf = it & 1;
    const float* const gh = sF;
    const float* const gl = sF + CH;
    const float* const wq = sF + 2 * CH;
    const float* const wk = sF + M::wk + buf * CH;

    if (it > 0) lds_barrier();  // the previous chunk's readers are done
    if constexpr (MODE != kAgg) tq.store(sQ);
    tk.store(sK);
    tv.store(sV);
    if constexpr (MODE == kOutFwdDg) tx.store(sX);
    lds_barrier();
    // this chunk's own waits come first in program order: the next chunk's
    // decays, and the loads that only this chunk uses
    issue_decay(REV ? c - 1 : c + 1, it + 1 < nch);
    f32x4_t cs[MODE == kOutRevDg ? MB : 1][MODE == kOutRevDg ? NB : 1], xv[MODE == kOutRevDg ? NB : 1][MODE == kOutRevDg ? NIB : 1];
    if constexpr (MODE == kOutRevDg) {
      const f32x4_t* p = chunk_state(c);
#pragma unroll
      for (int mb = 0; mb < MB; mb++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) cs[mb][nb] = p[(mb * NB + nb) * kThreads + threadIdx.x];
      const __amdgpu_buffer_rsrc_t rx = rows_rsrc(Xp + tb * r.ldx, r.ldx, nv, r.dn, sizeof(T));
#pragma unroll
      for (int nb = 0; nb < NB; nb++) {
        const int n = n0 + 16 * nb + 4 * g;
        const uint32_t vo = n < r.dn ? static_cast<uint32_t>((l15 * r.ldx + n) * sizeof(T)) : kOutside;
#pragma unroll
        for (int b = 0; b < NIB; b++) xv[nb][b] = load_rows(rx, vo + b * static_cast<uint32_t>(16 * r.ldx * sizeof(T)), Xp);
      }
    } else {
      issue(REV ? c - 1 : c + 1, it + 1 < nch);
    }
    const float wc = sF[M::wc + buf];

    f32x4_t Y[NB][NIB];
    if constexpr (MODE != kAgg) {
      // decayed scores of this wavefront's row block i, transposed: lane l
      // holds row i = l % 16 and four consecutive columns j
      const int ib = wave % NIB;
      const int i = 16 * ib + l15;
      const float ghi = gh[i], gli = gl[i];
      float rowsum = 0.0f;
#pragma unroll
      for (int jj = 0; jj < NIB / JW; jj++) {
        const int jb = jj * JW + wave / NIB;
        f32x4_t p{0.f, 0.f, 0.f, 0.f};
        float colsum[4] = {0.f, 0.f, 0.f, 0.f};
        if (REV ? jb >= ib : jb <= ib) {
          f32x4_t acc{0.f, 0.f, 0.f, 0.f};
          f32x4_t acx{0.f, 0.f, 0.f, 0.f};
          const int rj = 16 * jb + l15;
          if constexpr (kBf) {
#pragma unroll
            for (int kb = 0; kb < DM / 32; kb++)
              acc = mfma_bf16(load8(sK + at<T, DM>(rj, 32 * kb + 8 * g)), load8(sQ + at<T, DM>(i, 32 * kb + 8 * g)), acc);
          } else {
#pragma unroll
            for (int b = 0; b < DM / 16; b++) {
              const f32x4_t ka = load4(sK + at<T, DM>(rj, 16 * b + 4 * g)), qa = load4(sQ + at<T, DM>(i, 16 * b + 4 * g));
#pragma unroll
              for (int e = 0; e < 4; e++) acc = mfma_f32(ka[e], qa[e], acc);
            }
          }
          if constexpr (MODE == kOutFwdDg) {
            // the other pair's scores, X_i . V_j
            if constexpr (kBf) {
#pragma unroll
              for (int kb = 0; kb < DN / 32; kb++)
                acx = mfma_bf16(load8(sV + at<T, DN>(rj, 32 * kb + 8 * g)), load8(sX + at<T, DN>(i, 32 * kb + 8 * g)), acx);
            } else {
#pragma unroll
              for (int b = 0; b < DN / 16; b++) {
                const f32x4_t va = load4(sV + at<T, DN>(rj, 16 * b + 4 * g)), xa = load4(sX + at<T, DN>(i, 16 * b + 4 * g));
#pragma unroll
                for (int e = 0; e < 4; e++) acx = mfma_f32(va[e], xa[e], acx);
              }
            }
          }
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
        }
        store4(sP + at_p<T>(i, 16 * jb + 4 * g), p);
        if constexpr (MODE == kOutFwdDg) {
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float s = sum16(colsum[e]);
            if (l15 == 0) sCol[ib * CH + 16 * jb + 4 * g + e] = s;
          }
        }
      }
      if constexpr (MODE == kOutFwdDg) {
        rowsum = sum_groups(rowsum);
        if (g == 0) sRow[(wave / NIB) * CH + i] = rowsum;
      }

      if constexpr (MODE == kOutRevDg) {
        // the state entering this chunk meets the adjoint of the one leaving it
        float dot = 0.0f;
#pragma unroll
        for (int mb = 0; mb < MB; mb++)
#pragma unroll
          for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int e = 0; e < 4; e++) dot = fmaf(cs[mb][nb][e], S[mb][nb][e], dot);
        dot = sum_groups(sum16(dot));
        if (lane == 0) sDot[wave] = dot;
        issue(REV ? c - 1 : c + 1, it + 1 < nch);
      }

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
            const int q0 = at<T, DM>(16 * b + l15, 32 * kb + 4 * g), q1 = at<T, DM>(16 * b + l15, 32 * kb + 16 + 4 * g);
            qf[b] = __builtin_bit_cast(bf16x8_t, (Pair64{*reinterpret_cast<const uint2*>(sQ + q0),
                                                         *reinterpret_cast<const uint2*>(sQ + q1)}));
          }
#pragma unroll
          for (int nb = 0; nb < NB; nb++) {
            bf16x8_t hi, lo;
#pragma unroll
            for (int e = 0; e < 8; e++) {
              const float s = S[2 * kb + e / 4][nb][e % 4];
              hi[e] = static_cast<__bf16>(s);
              if constexpr (kDg) lo[e] = static_cast<__bf16>(s - static_cast<float>(hi[e]));
            }
#pragma unroll
            for (int b = 0; b < NIB; b++) {
              Y[nb][b] = mfma_bf16(hi, qf[b], Y[nb][b]);
              if constexpr (kDg) Y[nb][b] = mfma_bf16(lo, qf[b], Y[nb][b]);
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
#pragma unroll
      for (int b = 0; b < NIB; b++) {
        const float w = wq[16 * b + l15];
        float dot = 0.0f;
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
          Y[nb][b] = Y[nb][b] * w;
          if constexpr (MODE == kOutFwdDg) {
            const f32x4_t x = load4(sX + at<T, DN>(16 * b + l15, n0 + 16 * nb + 4 * g));
#pragma unroll
            for (int e = 0; e < 4; e++) dot = fmaf(x[e], Y[nb][b][e], dot);
          }
          if constexpr (MODE == kOutRevDg) {
            const f32x4_t x = xv[nb][b];
#pragma unroll
            for (int e = 0; e < 4; e++) dot = fmaf(x[e], Y[nb][b][e], dot);
          }
        }
        if constexpr (kDg) {
          dot = sum_groups(dot);
          if (g == 0) sRint[wave * CH + 16 * b + l15] = dot;
        }
      }
      if constexpr (MODE == kOutFwdDg) {
        // the state entering this chunk, for the reverse run
        f32x4_t* p = chunk_state(c);
#pragma unroll
        for (int mb = 0; mb < MB; mb++)
#pragma unroll
          for (int nb = 0; nb < NB; nb++) p[(mb * NB + nb) * kThreads + threadIdx.x] = S[mb][nb];
      }
    }
    if constexpr (MODE != kAgg) lds_barrier();  // scores and partial sums are in LDS; gh, gl, wq are free
    if (wave == kDecayWave && it + 1 < nch) decays(buf ^ 1);

    // V of this wavefront's columns, tokens along the lane's elements
    if constexpr (kBf) {
      bf16x8_t vf[CH / 32][NB];
#pragma unroll
      for (int kb = 0; kb < CH / 32; kb++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
          vf[kb][nb] = read_tr<DN>(sV, 32 * kb + 8 * g, n0 + 16 * nb, l15);
        }
      if constexpr (MODE != kAgg) {
#pragma unroll
        for (int b = 0; b < NIB; b++)
#pragma unroll
          for (int kb = 0; kb < CH / 32; kb++)
            if (REV ? 2 * kb + 1 >= b : 2 * kb <= b) {
              const bf16x8_t pf = load8(sP + at_p<T>(16 * b + l15, 32 * kb + 8 * g));
#pragma unroll
              for (int nb = 0; nb < NB; nb++) Y[nb][b] = mfma_bf16(vf[kb][nb], pf, Y[nb][b]);
            }
      }
      // the state's update
#pragma unroll
      for (int mb = 0; mb < MB; mb++)
#pragma unroll
        for (int nb = 0; nb < NB; nb++) S[mb][nb] = S[mb][nb] * wc;
#pragma unroll
      for (int kb = 0; kb < CH / 32; kb++) {
        const f32x4_t w0 = load4(wk + 32 * kb + 8 * g), w1 = load4(wk + 32 * kb + 8 * g + 4);
        bf16x8_t hi[NB], lo[NB];
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const float u = static_cast<float>(vf[kb][nb][e]) * (e < 4 ? w0[e % 4] : w1[e % 4]);
            hi[nb][e] = static_cast<__bf16>(u);
            lo[nb][e] = static_cast<__bf16>(u - static_cast<float>(hi[nb][e]));
          }
#pragma unroll
        for (int mb = 0; mb < MB; mb++) {
          const bf16x8_t kf = read_tr<DM>(sK, 32 * kb + 8 * g, 16 * mb, l15);
#pragma unroll
          for (int nb = 0; nb < NB; nb++) {
            S[mb][nb] = mfma_bf16(kf, hi[nb], S[mb][nb]);
            S[mb][nb] = mfma_bf16(kf, lo[nb], S[mb][nb]);
          }
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
    }
    if constexpr (MODE == kAgg) decay_seg *= wc;

    if constexpr (MODE != kAgg) {
      {
        const int64_t o0 = tb * r.ldo + h * r.dn;
        char* const ob = r.out ? static_cast<char*>(r.out) + o0 * es_out : nullptr;
        const __amdgpu_buffer_rsrc_t ro = rows_rsrc(ob, r.ldo, nv, r.dn, es_out);
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
          const int n = n0 + 16 * nb + 4 * g;
          const uint32_t vo = n < r.dn ? static_cast<uint32_t>((l15 * r.ldo + n) * es_out) : kOutside;
#pragma unroll
          for (int b = 0; b < NIB; b++) {
            const uint32_t v = vo + b * static_cast<uint32_t>(16 * r.ldo * es_out);
            store_rows(ro, v, Y[nb][b], static_cast<OT*>(nullptr));
          }
        }
      }
      // one lane per token: the decay gradient's sums inside the chunk
      if constexpr (kDg) {
        if (wave == kDecayWave) {
          double x = 0.0;
          if (lane < CH) {
            for (int w = 0; w < 4; w++) x += sRint[w * CH + lane];
            if constexpr (MODE == kOutFwdDg) {
              for (int w = 0; w < JW; w++) x += sRow[w * CH + lane];
              for (int w = 0; w < NIB; w++) x -= sCol[w * CH + lane];
            }
          }
          const int64_t o = (tb + lane) * a.Hv + h;
          if constexpr (MODE == kOutFwdDg) {
            // sums over i >= t
#pragma unroll
            for (int d = 1; d < CH; d <<= 1) {
              const double u = __shfl_down(x, d, 64);
              if (lane + d < CH) x += u;
            }
            if (lane < nv) r.tok[o] = static_cast<float>(x);
          } else {
            // sums over j < t
            x = prefix_sum(x) - x;
            if (lane < nv) {
              const float dot = (sDot[0] + sDot[1]) + (sDot[2] + sDot[3]);
              const double dg = x + static_cast<double>(wc * dot) + static_cast<double>(r.tok[o]);
              if (r.dg_tok) r.dg_tok[o] = static_cast<float>(dg);
              dg_sum += dg;
            }
          }
        }
      }
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
#pragma unroll
    for (int mb = 0; mb < MB; mb++)
#pragma unroll
      for (int nb = 0; nb < NB; nb++) {
        const int m = 16 * mb + 4 * g, n = n0 + 16 * nb + l15;
        if (m < r.dm && n < r.dn)
#pragma unroll
          for (int e = 0; e < 4; e++) s_out[(m + e) * r.sm + n * r.sn] = S[mb][nb][e];
      }
  }
  if constexpr (MODE == kOutRevDg) {
    if (r.dg_seg && wave == kDecayWave) {
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) dg_sum += __shfl_xor(dg_sum, d, 64);
      if (lane == 0) r.dg_seg[static_cast<int64_t>(slot) * a.Hv + h] = dg_sum;
    }
  }
}

// Kinds: kGrad... with PT the type of dq and dk, float where the value heads
// of a key head are summed afterwards.
template <class T, class PT, int DK, int DV, int KIND>
__global__ __launch_bounds__(kThreads, 2) void k_linattn(Args a) {
  extern __shared__ __attribute__((aligned(16))) char smem_la[];
  if constexpr (KIND == kForward) {
    run<T, T, DK, DV, false, kOut>(a, a.run[0], smem_la);
  } else if constexpr (KIND == kAggregate) {
    if (blockIdx.z == 0) run<T, T, DK, DV, false, kAgg>(a, a.run[0], smem_la);
    else run<T, T, DK, DV, true, kAgg>(a, a.run[1], smem_la);
  } else if constexpr (KIND == kGradFirst) {
    if (blockIdx.z == 0) run<T, PT, DV, DK, false, kOutFwdDg>(a, a.run[0], smem_la);
    else run<T, T, DK, DV, true, kOut>(a, a.run[1], smem_la);
  } else if constexpr (KIND == kGradSecond) {
    run<T, PT, DV, DK, true, kOutRevDg>(a, a.run[0], smem_la);
  } else {
    if (blockIdx.z == 0) run<T, PT, DV, DK, false, kOut>(a, a.run[0], smem_la);
    else if (blockIdx.z == 1) run<T, T, DK, DV, true, kOut>(a, a.run[1], smem_la);
    else run<T, PT, DV, DK, true, kOut>(a, a.run[2], smem_la);
  }
}

constexpr int max2(int a, int b) { return a > b ? a : b; }

template <class T, int DK, int DV, int KIND>
constexpr int lds_bytes() {
  if (KIND == kForward) return Lds<T, DK, DV, kOut>::bytes;
  if (KIND == kAggregate) return Lds<T, DK, DV, kAgg>::bytes;
  if (KIND == kGradFirst) return max2(Lds<T, DV, DK, kOutFwdDg>::bytes, Lds<T, DK, DV, kOut>::bytes);
  if (KIND == kGradSecond) return Lds<T, DV, DK, kOutRevDg>::bytes;
  return max2(Lds<T, DV, DK, kOut>::bytes, Lds<T, DK, DV, kOut>::bytes);
}

template <class T, class PT, int DK, int DV, int KIND>
hipError_t launch_one(const Args& a, int nz, hipStream_t st) {
  constexpr int lds = lds_bytes<T, DK, DV, KIND>();
  static_assert(lds <= 80 * 1024, "two workgroups share a CU's 160 KB");
  auto kern = k_linattn<T, PT, DK, DV, KIND>;
  if constexpr (lds > 64 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(slot_count(a.sq.T, a.sq.S, a.sq.L)), static_cast<unsigned>(a.Hv),
                  static_cast<unsigned>(nz));
  kern<<<grid, kThreads, lds, st>>>(a);
  return hipGetLastError();
}

template <class T, class PT, int DK, int DV>
hipError_t launch_grad(Kernel k, const Args& a, int nz, hipStream_t st) {
  if (k == kGradFirst) return launch_one<T, PT, DK, DV, kGradFirst>(a, nz, st);
  if (k == kGradSecond) return launch_one<T, PT, DK, DV, kGradSecond>(a, nz, st);
  return launch_one<T, PT, DK, DV, kGradPlain>(a, nz, st);
}

template <class T, int DK, int DV>
hipError_t launch_kind(Kernel k, const Args& a, int nz, hipStream_t st) {
  if (k == kForward) return launch_one<T, T, DK, DV, kForward>(a, nz, st);
  if (k == kAggregate) return launch_one<T, T, DK, DV, kAggregate>(a, nz, st);
  if (a.sum_heads) return launch_grad<T, float, DK, DV>(k, a, nz, st);
  return launch_grad<T, T, DK, DV>(k, a, nz, st);
}

}  // namespace

}  // namespace la
