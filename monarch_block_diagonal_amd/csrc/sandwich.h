// Sandwich norm (internal): what the planning (sandwich.hip) hands to the
// kernels (sandwich_kernels.h, compiled for each type on its own).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace monarch {

constexpr int64_t kSandwichCus = 256;
constexpr int kSandwichMaxFeatures = 16384;   // 1024 threads x 4 pieces of 4 fp32 elements

// Threads of a team and pieces of 16 bytes that each holds of a row.
struct Shape {
  int team, pieces;
};
Shape sandwich_fwd_shape(int64_t d, bool bf16);

struct SandwichFwd {
  const void *h, *y, *post_w, *post_b, *gate, *pre_w, *pre_b;
  void *h_out, *n_out;
  float* stats;
  uint32_t* low;   // bits that h_out's rounding to bf16 left, a word a piece (low_bits); null: not kept
  int64_t rows, rows_per_gate;
  int d, post, pre;
  float skip, branch, eps;
};

// How the rows of a backward call are cut (GATE). CHUNK: chunk c holds rows of one
// gate row only (chunk / cpg), and its sums are of D alone; the gate and the
// branch scale are applied when the chunks are joined. RUN: many gate runs, or
// short ones where cutting them does not pay; each is summed by one team, which
// stores its dgate row itself, and the chunk's sums are of g * D. TOKEN: RUN with one row a run.
enum { CHUNK = 0, RUN = 1, TOKEN = 2 };

struct SandwichBwd {
  const void *dh_out, *dn, *h_out, *y;
  const float* stats;
  const uint32_t* low;   // as for the forward pass; where nothing is kept, any address
  int low_row;           // words a row; 0: h_out is taken as it is
  const void *post_w, *post_b, *gate, *pre_w, *pre_b;
  void *dh, *dy, *dgate;
  float* part;          // [chunks][sums][d]
  int64_t rows, rows_per_gate, chunk_rows, cpg;
  int d, post, pre, sums;
  int s_post, s_postb, s_pre, s_preb;   // index of each sum in a chunk, -1: not taken
  float skip, branch;
};

struct SandwichBwdPlan {
  Shape shape;
  int gate;      // CHUNK, RUN or TOKEN
  bool bias;
  int64_t chunks, chunk_rows, cpg, rows_per_gate;
  int sums, s_post, s_postb, s_pre, s_preb;
  size_t ws;
};

// Joins the chunks' sums. A job is one output row: the weight gradients (sums
// over every chunk, weighted by the chunk's gate row) and, when chunks hold
// sums of D alone, one dgate row each. A workgroup takes 32 columns; 32 slices
// of 32 threads sum contiguous chunk ranges, and the slices are added in order.
// Bound by latency: 16 loads of a slice, eight at a time; 4.0 us for 512 chunks of
// 768 columns and 16 gates (15 us with 64 columns x 16 slices).
struct SandwichJoin {
  const float* part;
  const void *gate, *post_w, *post_b;   // gate: null where the sums hold it already
  void *dgate, *dpost_w, *dpost_b, *dpre_w, *dpre_b;
  int chunks, cpg, d, sums, s_post, s_postb, s_pre, s_preb;
  float branch;
};
constexpr int kWeightJobs = 4;   // post_w, post_b, pre_w, pre_b; then one job a gate row

// T: float, or uint16_t for bfloat16.
template <typename T> hipError_t sandwich_launch_fwd(const SandwichFwd& a, hipStream_t s);
template <typename T>
hipError_t sandwich_launch_bwd(const SandwichBwd& a, const SandwichBwdPlan& p, hipStream_t s);
template <typename T>
hipError_t sandwich_launch_join(const SandwichJoin& a, int64_t jobs, hipStream_t s);

}  // namespace monarch
