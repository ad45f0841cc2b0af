// linattn_seqs.hpp -- device-side lookup of segments and chunks of packed
// sequences (see Seqs in linattn.hpp).
#pragma once

#include "linattn.hpp"

namespace la {

struct Segment {
  int32_t seq;
  int32_t t0, t1;      // its tokens
  int32_t chunk_slot;  // of its first chunk
  bool first, last;    // of its sequence
};

// The segment of a slot; false if the slot has none.  The sequence is found
// by bisection over the first slots start[s] / L + s, which increase with s.
inline __device__ bool find_segment(const Seqs& sq, uint32_t slot, int ch, Segment* o) {
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

// Every kAnchor-th chunk of a segment, counted from its last one, is an
// anchor: the runs of the gradient keep the states there.  Anchors own slots
// as segments do.
inline __device__ int64_t anchor_slot(const Segment& s, uint32_t slot) { return s.chunk_slot / kAnchor + slot; }

// 2^x of a 64-bit x, to fp32 accuracy also for large |x|.
__device__ __forceinline__ float exp2_split(double x) {
  const float h = static_cast<float>(x);
  const float l = static_cast<float>(x - static_cast<double>(h));
  const float e = __builtin_amdgcn_exp2f(h);
  return fmaf(e, l * 0.69314718055994531f, e);
}

// A log decay in base 2 and 64 bits.  One below e^-13000 is taken as that:
// both are zero in every product, and -inf would make a NaN of inf - inf.
__device__ __forceinline__ double decay_log2(float g) {
  return static_cast<double>(g < -13000.0f ? -13000.0f : g) * 1.4426950408889634;
}

}  // namespace la
