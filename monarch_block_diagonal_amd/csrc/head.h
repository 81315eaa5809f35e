// The head loss's launches (internal): planning and C entries in head.hip, the
// products in head_gemm.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_pipe.h"

namespace monarch {

constexpr int64_t kThinRows = 32;    // rows that HEAD_THIN takes
constexpr int64_t kHeadRows = 256;   // rows of the workspace's copies are a multiple of this, and so are a piece's columns

// Workgroups of a launch, so that it has fewer than 2^32 threads (workgroups have 512 at most), which is all that
// a launch can have. Calls of more rows or words than that launch a kernel several times.
constexpr int64_t kLaunchGroups = int64_t(1) << 22;

// f(first, grid) launches the workgroups [first, first + grid).
template <class F>
hipError_t launch_groups(int64_t groups, F f) {
  for (int64_t first = 0; first < groups; first += kLaunchGroups) {
    const int64_t n = groups - first < kLaunchGroups ? groups - first : kLaunchGroups;
    f(first, dim3(static_cast<unsigned>(n)));
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

// What the products' epilogues take of a row: its largest logit and the factors of
// its exponentials; the label's share is taken off at the label.
struct HeadRow {
  float m, a, b, off;   // g = a 2^((z - m) ct) + b 2^((z - m) log2 e) - off [v = label]
};

// The labels' softmax beside the teacher's at T.
enum HeadSecond {
  HEAD_ONE = 0,     // none, or T = 1: one softmax
  HEAD_OWN = 1,     // exponentials of its own
  HEAD_SQUARE = 2   // T = 2: e^z is the square of e^(z/2)
};

// A finite value's nearest that is finite in bf16 too (the largest ones of fp32 round to infinity).
__device__ __forceinline__ float finite_bf16(float v) {
  constexpr float kMost = 3.38953138925153547590e38f;
  return isfinite(v) ? __builtin_amdgcn_fmed3f(v, -kMost, kMost) : v;
}

// g of one logit; operations and roundings are the same wherever it is computed.
template <int SECOND>
__device__ __forceinline__ float head_g(const HeadRow& r, float logit, float ct, bool label) {
#pragma clang fp contract(off)
  const float z = logit - r.m, e = __builtin_amdgcn_exp2f(z * ct);
  float g = r.a * e;
  if constexpr (SECOND == HEAD_OWN) g = fmaf(r.b, __builtin_amdgcn_exp2f(z * 1.44269504088896340736f), g);
  if constexpr (SECOND == HEAD_SQUARE) g = fmaf(r.b * e, e, g);
  return label ? g - r.off : g;
}

// HEAD_THIN: logits of at most 32 rows; HEAD_32: these in fp32 where words are no whole pieces, and dx in bf16
enum HeadShape { HEAD_256 = 0, HEAD_128 = 1, HEAD_32 = 2, HEAD_THIN = 3 };

struct HeadLogits {
  PipeProduct pr;             // A: the head's words, B: the rows
  const float* raw;           // fp32, HEAD_THIN: the head itself [vocab][d]
  const int* count;           // rows in use
  int f32;                    // operands are fp32, as three planes
  int64_t vocab, v0, v1;      // words of this launch: [v0, v1)
  int64_t d;                  // k
  int64_t rows, np;           // rows of the call, and of the workspace's copies
  float ct;                   // log2(e) / temperature
  const int* label;           // a row: its label, -1 without one
  // sums: part [tiles of words][np][3] (largest logit, sum at T, sum at 1), z of the label
  float* part;
  float* z_label;
  float* z;                   // HEAD_THIN, or null: the logits [rows][vp]
  // gradient: g [planes][np][vp]
  const HeadRow* row;
  uint16_t* g;
  float* few;                 // fp32, few rows: g as it is, [kThinRows][vp]
  int64_t vp, g_plane;
  int fold;                   // bf16, few rows: g has two parts, the second one's rows `fold` behind the first's; or 0
};

struct HeadDx {
  PipeProduct pr;             // A: the head's words [v][d], B: g [n][v]
  const int* count;           // rows of g in use
  int f32;
  int64_t d, dp, np;
  int64_t k, chunk;           // words of this piece, words a split
  int splits;
  float* part;                // [splits][np][dp]
  int add;                    // whether a piece before has written part
  int64_t dt, nt;             // tiles (set by the launch)
};

struct HeadDw {
  PipeProduct pr;             // A: the rows [n][d], B: g [n][v]
  const int* count;
  int f32;
  const float* scale;         // what g was divided by (bf16)
  int64_t d, dp, cols;        // cols: words of this piece
  int splits;
  float* part;                // [splits][cols][dp], or null:
  void* dw;                   // the piece's first word of dw [vocab][d]
  int64_t dt, vt;             // tiles (set by the launch)
};

int64_t head_tile_words(HeadShape s, int64_t vocab);    // words behind one of a logits launch's sums
int64_t head_tile_rows(HeadShape s);     // rows of a logits and a dx tile
int64_t head_tile_features(HeadShape s); // features of a dx tile
hipError_t head_launch_sums(const HeadLogits& a, HeadShape s, HeadSecond second, hipStream_t st);
hipError_t head_launch_grad(const HeadLogits& a, HeadShape s, HeadSecond second, hipStream_t st);
// dx and dw of a piece (HEAD_32: dx's tiles have 64 rows of g, dw's are HEAD_128's)
hipError_t head_launch_products(const HeadDx& x, const HeadDw& w, HeadShape s, hipStream_t st);

// Both products of at most kThinRows rows in fp32.
struct HeadFew {
  const float* g;             // [kThinRows][vp]
  int64_t vp;
  const float* x;             // rows idx[k] for k < *count
  int64_t ldx;
  const int *idx, *count;
  const float* w;             // the piece's words
  float *dw, *part;           // part [splits][head_few_rows][dp]
  int64_t d, dp, words;
  bool add;                   // part already holds other pieces' sums
};
int64_t head_few_rows(int64_t rows);
// words of a split for a piece of `words`
int64_t head_few_run(int64_t rows, int64_t d, int64_t words);
hipError_t head_launch_few(const HeadFew& a, int64_t rows, int64_t run, int64_t splits, hipStream_t st);

}  // namespace monarch
