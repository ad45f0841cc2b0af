// linattn.hpp -- internal launch interface of the decayed linear attention
// (kernels in linattn.inl, instantiated by the linattn_*.hip files; the C
// entries are in linattn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace la {

// Where the tokens are: S packed sequences of a T-row array, cut into segments
// of L tokens (a multiple of the chunk).  Sequence s owns the segment slots
// start[s] / L + s ..: slots of different sequences are disjoint (an empty
// sequence still has one), and there are T / L + S of them.  Its chunks own
// chunk slots in the same way.
struct Seqs {
  int64_t T;
  int32_t S;
  const int32_t* start;  // [S + 1] or null: S sequences of T / S tokens
  int64_t L;
};

inline __host__ __device__ int64_t slot_count(int64_t T, int32_t S, int64_t L) { return T / L + S; }

// One linear attention over all segments: out_i = qs sum_j decay(i, j)
// (Q_i . K_j) V_j ks + the state's part, forward in time (j <= i) or in
// reverse (j >= i).  The state is sum_j decay K_j V_j^T, dm x dn.
struct Run {
  const void *Q, *K, *V, *X;       // token rows; X: the operand of the decay gradient's dot
  int64_t ldq, ldk, ldv, ldx, ldo;
  int32_t gq, gk, gv;              // value heads per head of Q, K and V (X has V's)
  int32_t dm, dn;
  float qs, ks;
  const float* s0;                 // [S][Hv] states at the sequences' ends, or null (zero)
  float* seg;                      // [slots][Hv] states entering each segment, or null (one segment each)
  float* seg_decay;                // [slots][Hv] product of a segment's decays (aggregate pass)
  float* s_end;                    // [S][Hv] the state leaving the sequences, or null
  int32_t sm, sn;                  // strides of a state's dm and dn index
  void* out;                       // token rows of Hv heads, or null
  float* tok;                      // [Hv][T] sums inside the chunk of the decay gradient's terms
  float* anchors;                  // [anchor slots][Hv][dm][dn] (padded) states kept for it
};

struct Args {
  Seqs sq;
  int32_t Hv, dkdv;                // heads, floats of a state
  const float* log_decay;
  int64_t ld_decay;                // Hv, or 0 for one decay per head
  int32_t sum_heads;               // dq and dk are float32, one per value head
  int32_t nz;                      // runs of the launch,
  int32_t run_of[3];               // and which they are
  uint32_t units;                  // segment slots x heads
  Run run[3];
};

enum Kernel {
  kForward,    // run 0: y
  kForwardState,  // the same where the final state is an output too
  kAggregate,  // run 0: the segments' state sums, forward in time; run 1: in reverse
  kAggregateOut,  // the same where the states reach only outputs of the io type
  kGradPlain,  // runs 0, 1, 2: dq, dk (and the adjoint of h0), dv
  kGradDecay   // the same with the decay gradient's terms
};

constexpr int kAnchor = 8;  // chunks between kept states

// Tokens of a chunk: 64 for bf16, 32 for fp32 (the same LDS bytes a tile).
constexpr int chunk_tokens(bool bf16) { return bf16 ? 64 : 32; }

// Padded head width the kernels are built for.
inline int padded(int d) { return d <= 64 ? 64 : 128; }

// Floats of one padded state.
inline int64_t state_floats(int dk, int dv) { return static_cast<int64_t>(padded(dk)) * padded(dv); }

// One launch over every segment slot, head and run, by io type and padded dk.
hipError_t launch_bf16_64(Kernel k, int dv, const Args& a, hipStream_t st);
hipError_t launch_bf16_128(Kernel k, int dv, const Args& a, hipStream_t st);
hipError_t launch_f32_64(Kernel k, int dv, const Args& a, hipStream_t st);
hipError_t launch_f32_128(Kernel k, int dv, const Args& a, hipStream_t st);

}  // namespace la
