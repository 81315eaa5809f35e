// Sandwich norm: planning and C entries. The formulas and the kernels are in
// sandwich_kernels.h.
#include "sandwich.h"

#include <math.h>

#include <initializer_list>

#include "api_internal.h"
#include "monarch.h"

namespace monarch {
namespace {

constexpr int64_t kLimit = int64_t(1) << 31;
// gate rows where there are no rows: each is a workgroup of the join
constexpr int64_t kEmptyGates = int64_t(1) << 21;

// The smallest team whose threads hold at most `few` (up to a wave) or `many`
// pieces of a row; `last` for any row that is wider.
Shape shape_of(int64_t d, bool bf16, int first, int last, int few, int many) {
  const int per = bf16 ? 8 : 4;
  const int64_t pieces = (d + per - 1) / per;
  int t = first;
  while (t < last && (pieces + t - 1) / t > (t > 64 ? many : few)) t *= 2;
  return {t, static_cast<int>((pieces + t - 1) / t)};
}

Shape bwd_shape(int64_t d, bool bf16) {
  return shape_of(d, bf16, 32, bf16 ? 512 : 1024, bf16 ? 3 : 4, bf16 ? 2 : 4);
}

constexpr int64_t kRunRows = 32;   // gate runs up to this long may be a team's own however few there are

// Whether short gate runs are cut into chunks: where the rows that one team would take
// in turn cost more than joining the gate rows' sums does. Both are fitted to
// measured crossovers (runs of 2 to 32 rows, 64 to 16384 features, both types): a row 0.75
// us and 45 ns an element of a thread, three times that for rows whose sums take their
// CU's LDS; joining 30 ns a gate row and 3 ns a workgroup of 32 columns. Of 458 drawn
// sizes 9 came out more than 15% slower than the other way would have (70% at most).
// Backward and join, cut against whole: 64 x 768 bf16 with 2 gates 9 / 76 us, 16384 x
// 768 with 512 gates 73 / 91, with 2048 gates 204 / 40; 256 x 16384 with 8 gates 46 / 326.
bool cut_short_runs(int64_t rows_per_gate, int64_t d, int64_t gates, const Shape& s, bool wide, bool bf16) {
  const int64_t row = (750 + 45 * s.pieces * (bf16 ? 8 : 4)) * (wide ? 3 : 1);
  return gates * (30 + 3 * ((d + 31) / 32)) < rows_per_gate * row;
}

// Everything about a backward call that depends on sizes alone (`with`: which
// of post_w, post_b, gate, pre_w, pre_b there are, as the sums they need).
SandwichBwdPlan bwd_plan(int64_t rows, int64_t d, int64_t gates, bool has_y, bool post_bias, bool has_pre,
                 bool pre_bias, bool bf16) {
  SandwichBwdPlan p = {};
  p.shape = bwd_shape(d, bf16);
  p.bias = post_bias || pre_bias;
  p.rows_per_gate = gates > 0 ? rows / gates : rows;
  const int teams = p.shape.team > 64 ? 1 : 256 / p.shape.team;
  // workgroups aimed at: two a CU, one where the sums of a wide row take its LDS
  const bool wide = p.shape.team * p.shape.pieces * (bf16 ? 8 : 4) > 8192;
  const int64_t aim = kSandwichCus * (wide ? 1 : 2);
  // a gate run is a team's own where there are enough of them for every team, or where
  // it is short and cutting it does not pay
  const bool own = gates >= aim * teams ||
                   (p.rows_per_gate <= kRunRows && !cut_short_runs(p.rows_per_gate, d, gates, p.shape, wide, bf16));
  p.gate = rows == 0 || gates <= 1 ? CHUNK : p.rows_per_gate == 1 ? TOKEN : own ? RUN : CHUNK;
  if (rows == 0) {
    p.cpg = 0;   // no chunk: every sum is empty
  } else if (p.gate != CHUNK) {
    const int64_t units = gates, slots = aim * teams;
    p.chunk_rows = (units + slots - 1) / slots;
    p.chunks = (units + p.chunk_rows * teams - 1) / (p.chunk_rows * teams);
    p.cpg = 1;
  } else {
    const int64_t g = gates > 0 ? gates : 1;
    int64_t cpg = (aim + g - 1) / g;
    const int64_t most = (p.rows_per_gate + teams - 1) / teams;
    if (cpg > most) cpg = most;
    p.chunk_rows = (p.rows_per_gate + cpg - 1) / cpg;
    p.cpg = (p.rows_per_gate + p.chunk_rows - 1) / p.chunk_rows;
    p.chunks = g * p.cpg;
  }
  int n = 0;
  p.s_post = has_y ? n++ : -1;
  p.s_postb = has_y && post_bias ? n++ : -1;
  p.s_pre = has_pre ? n++ : -1;
  p.s_preb = has_pre && pre_bias ? n++ : -1;
  p.sums = n;
  p.ws = (static_cast<size_t>(p.chunks) * n * d * sizeof(float) + 255) / 256 * 256;
  return p;
}

int check_sizes(int64_t rows, int64_t d, int64_t gates, int post, int pre, int dtype) {
  if (dtype != MONARCH_F32 && dtype != MONARCH_BF16) return MONARCH_ERR_DTYPE;
  if (post < MONARCH_NORM_NONE || post > MONARCH_NORM_LAYER || pre < MONARCH_NORM_NONE ||
      pre > MONARCH_NORM_LAYER)
    return MONARCH_ERR_DTYPE;
  if (rows < 0 || rows >= kLimit || d <= 0 || d > kSandwichMaxFeatures || gates < 0) return MONARCH_ERR_SHAPE;
  if (gates > (rows > 0 ? rows : kEmptyGates) || (gates > 0 && rows % gates != 0)) return MONARCH_ERR_SHAPE;
  return MONARCH_OK;
}

// Whether the forward pass keeps what h_out's rounding left, for the backward pass:
// behind the statistics, a word for 8 elements.
bool keeps_low(const void* y, int pre, bool bf16) { return y && pre != MONARCH_NORM_NONE && bf16; }

bool any_misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (misaligned(p)) return true;
  return false;
}

}  // namespace

Shape sandwich_fwd_shape(int64_t d, bool bf16) {
  return shape_of(d, bf16, 16, 1024, bf16 ? 3 : 4, bf16 ? 2 : 4);
}

}  // namespace monarch

using namespace monarch;

extern "C" {

int monarch_sandwich_fwd(const void* h, const void* y, const void* post_w, const void* post_b,
                         const void* gate, const void* pre_w, const void* pre_b, void* h_out,
                         void* n_out, void* stats, int64_t rows, int64_t features, int64_t gates,
                         int post_norm, int pre_norm, float skip_scale, float branch_scale,
                         float eps, int dtype, void* stream, void* const* events, int n_events) {
  int st = check_sizes(rows, features, gates, post_norm, pre_norm, dtype);
  if (st) return st;
  if (!(eps >= 0.0f) || !isfinite(eps) || !isfinite(skip_scale) || !isfinite(branch_scale))
    return MONARCH_ERR_VALUE;
  if (gates > 0 && !gate) return MONARCH_ERR_NULL;
  if (rows > 0) {
    if (!h || !stats || (y && !h_out) || (pre_norm != MONARCH_NORM_NONE && !n_out))
      return MONARCH_ERR_NULL;
  }
  if (any_misaligned({h, y, post_w, post_b, gate, pre_w, pre_b, h_out, n_out, stats}))
    return MONARCH_ERR_ALIGN;
  if (rows == 0) return MONARCH_OK;
  SandwichFwd a;
  a.h = h, a.y = y, a.post_w = post_w, a.post_b = post_b, a.gate = gates > 0 ? gate : nullptr;
  a.pre_w = pre_w, a.pre_b = pre_b, a.h_out = h_out, a.n_out = n_out;
  a.stats = static_cast<float*>(stats);
  a.low = keeps_low(y, pre_norm, dtype == MONARCH_BF16) ? static_cast<uint32_t*>(stats) + rows * 4 : nullptr;
  a.rows = rows, a.rows_per_gate = gates > 0 ? rows / gates : rows;
  a.d = static_cast<int>(features), a.post = post_norm, a.pre = pre_norm;
  a.skip = skip_scale, a.branch = branch_scale, a.eps = eps;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Tracer tr{events, n_events, 0, s};
  st = record_hip(tr.mark());
  if (st) return st;
  st = record_hip(dtype == MONARCH_BF16 ? sandwich_launch_fwd<uint16_t>(a, s)
                                         : sandwich_launch_fwd<float>(a, s));
  if (st) return st;
  return record_hip(tr.mark());
}

size_t monarch_sandwich_stats_bytes(int64_t rows, int64_t features, int with_y, int pre_norm, int dtype) {
  if (check_sizes(rows, features, 0, 0, pre_norm, dtype)) return 0;
  const bool low = keeps_low(with_y ? &with_y : nullptr, pre_norm, dtype == MONARCH_BF16);
  return static_cast<size_t>(rows) * (4 + (low ? (features + 7) / 8 : 0)) * sizeof(float);
}

size_t monarch_sandwich_bwd_workspace_bytes(int64_t rows, int64_t features, int64_t gates,
                                            int with_bias, int dtype) {
  if (check_sizes(rows, features, gates, 0, 0, dtype) || rows == 0) return 0;
  return bwd_plan(rows, features, gates, true, with_bias != 0, true, with_bias != 0,
                  dtype == MONARCH_BF16)
      .ws;
}

int monarch_sandwich_bwd(const void* dh_out, const void* dn, const void* h_out, const void* y,
                         const void* stats, const void* post_w, const void* post_b,
                         const void* gate, const void* pre_w, const void* pre_b, void* dh, void* dy,
                         void* dpost_w, void* dpost_b, void* dgate, void* dpre_w, void* dpre_b,
                         void* workspace, size_t workspace_bytes, int64_t rows, int64_t features,
                         int64_t gates, int post_norm, int pre_norm, float skip_scale,
                         float branch_scale, int dtype, void* stream, void* const* events,
                         int n_events) {
  int st = check_sizes(rows, features, gates, post_norm, pre_norm, dtype);
  if (st) return st;
  if (!isfinite(skip_scale) || !isfinite(branch_scale)) return MONARCH_ERR_VALUE;
  const bool has_pre = pre_norm != MONARCH_NORM_NONE, bf16 = dtype == MONARCH_BF16;
  if (gates > 0 && !gate) return MONARCH_ERR_NULL;
  if (rows > 0) {
    if (!stats || !dh || (y && !dy) || (has_pre && (!dn || !h_out)) || (!has_pre && !dh_out))
      return MONARCH_ERR_NULL;
  }
  if (any_misaligned({dh_out, dn, h_out, y, stats, post_w, post_b, gate, pre_w, pre_b, dh, dy,
                      dpost_w, dpost_b, dgate, dpre_w, dpre_b, workspace}))
    return MONARCH_ERR_ALIGN;
  if (rows > 0 && !y && (dy || dpost_w || dpost_b || dgate)) return MONARCH_ERR_NULL;
  if ((dpost_w && !post_w) || (dpost_b && !post_b) || (dgate && gates == 0) ||
      (dpre_w && !(has_pre && pre_w)) || (dpre_b && !(has_pre && pre_b)))
    return MONARCH_ERR_NULL;
  const SandwichBwdPlan p = bwd_plan(rows, features, gates, y || rows == 0, post_b != nullptr, has_pre,
                             pre_b != nullptr, bf16);
  if (rows > 0 && p.ws > 0 && !workspace) return MONARCH_ERR_NULL;
  if (rows > 0 && workspace_bytes < p.ws) return MONARCH_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Tracer tr{events, n_events, 0, s};
  if (rows > 0) {
    SandwichBwd a;
    a.dh_out = dh_out, a.dn = dn, a.h_out = h_out, a.y = y;
    a.stats = static_cast<const float*>(stats);
    a.low_row = keeps_low(y, pre_norm, bf16) ? static_cast<int>((features + 7) / 8) : 0;
    a.low = static_cast<const uint32_t*>(stats) + (a.low_row ? rows * 4 : 0);
    a.post_w = post_w, a.post_b = post_b, a.gate = gates > 0 ? gate : nullptr;
    a.pre_w = has_pre ? pre_w : nullptr, a.pre_b = has_pre ? pre_b : nullptr;
    a.dh = dh, a.dy = dy, a.dgate = dgate, a.part = static_cast<float*>(workspace);
    a.rows = rows, a.rows_per_gate = p.rows_per_gate, a.chunk_rows = p.chunk_rows, a.cpg = p.cpg;
    a.d = static_cast<int>(features), a.post = post_norm, a.pre = pre_norm, a.sums = p.sums;
    a.s_post = p.s_post, a.s_postb = p.s_postb, a.s_pre = p.s_pre, a.s_preb = p.s_preb;
    a.skip = skip_scale, a.branch = branch_scale;
    st = record_hip(tr.mark());
    if (st) return st;
    st = record_hip(bf16 ? sandwich_launch_bwd<uint16_t>(a, p, s) : sandwich_launch_bwd<float>(a, p, s));
    if (st) return st;
  }
  if (dpost_w || dpost_b || dgate || dpre_w || dpre_b) {
    SandwichJoin j;
    j.part = static_cast<const float*>(workspace);
    j.gate = gates > 0 && p.gate == CHUNK ? gate : nullptr;
    j.post_w = post_w, j.post_b = post_b;
    j.dgate = dgate, j.dpost_w = dpost_w, j.dpost_b = dpost_b, j.dpre_w = dpre_w, j.dpre_b = dpre_b;
    j.chunks = static_cast<int>(p.chunks), j.cpg = static_cast<int>(p.cpg);
    j.d = static_cast<int>(features), j.sums = p.sums;
    j.s_post = p.s_post, j.s_postb = p.s_postb, j.s_pre = p.s_pre, j.s_preb = p.s_preb;
    j.branch = branch_scale;
    const int64_t jobs = kWeightJobs + (dgate && p.gate == CHUNK ? gates : 0);
    st = record_hip(tr.mark());
    if (st) return st;
    st = record_hip(bf16 ? sandwich_launch_join<uint16_t>(j, jobs, s)
                         : sandwich_launch_join<float>(j, jobs, s));
    if (st) return st;
  }
  return record_hip(tr.mark());
}

int monarch_sandwich_describe(int direction, int64_t rows, int64_t features, int64_t gates,
                              int dtype, char* buf, size_t buf_len) {
  const int st = check_sizes(rows, features, gates, 0, 0, dtype);
  if (st) return st;
  if (direction != 0 && direction != 1) return MONARCH_ERR_DTYPE;
  static const char* const fwd[] = {"sandwich_fwd"};
  static const char* const bwd[] = {"sandwich_bwd", "sandwich_join"};
  if (direction == 0) return write_names(fwd, rows > 0 ? 1 : 0, buf, buf_len);
  return rows > 0 ? write_names(bwd, 2, buf, buf_len) : write_names(bwd + 1, 1, buf, buf_len);
}

}  // extern "C"
