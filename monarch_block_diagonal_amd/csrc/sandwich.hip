// Sandwich norm: the norm after a block, its gate, the scaled residual join
// and the norm before the next block, forward and backward.
//
//   u  = norm_post(y) * w_post + b_post
//   h' = skip * h + branch * g * u
//   n  = norm_pre(h') * w_pre + b_pre
//
// norm(v) = (v - mu) * rho with rho = 1/sqrt(mean((v - mu)^2) + eps), mu the mean
// (LAYER) or 0 (RMS), and v itself without a norm. The gate g [gates, d]
// holds one row for rows/gates consecutive rows. With q = dn * w_pre,
// hhat = (h' - mu) rho and yhat likewise, the gradients are
//   D  = dh' + rho (q - hhat mean(q hhat) - [LAYER] mean(q)),   dh = skip D
//   e  = branch g D, q2 = e w_post
//   dy = rho (q2 - yhat mean(q2 yhat) - [LAYER] mean(q2))
//   dg = branch sum D u, dw_post = sum e yhat, db_post = sum e,
//   dw_pre = sum dn hhat, db_pre = sum dn      (sums over rows).
//
// A row is held in registers by a team of threads (team.h): every tensor is
// read once and written once. All arithmetic and all sums are fp32; results
// are rounded once, at their store. n is computed from h' before its rounding.
#include <math.h>

#include <initializer_list>

#include "api_internal.h"
#include "monarch.h"
#include "team.h"

namespace monarch {
namespace {

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int kMaxFeatures = 16384;   // 1024 threads x 4 pieces of 4 fp32 elements

struct SandwichFwd {
  const void *h, *y, *post_w, *post_b, *gate, *pre_w, *pre_b;
  void *h_out, *n_out;
  float* stats;
  int64_t rows, rows_per_gate;
  int d, post, pre;
  float skip, branch, eps;
};

template <typename T, int N>
__device__ __forceinline__ void load_or(const void* p, int64_t off, int at, int d, float fill,
                                        float (&v)[N]) {
  if (p) {
    PieceOf<T>::unpack(load_piece<T>(static_cast<const T*>(p) + off, at, d), v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = fill;
  }
}

// mean and 1/sqrt(mean square about it + eps) of the team's row (zero past d)
template <int TEAM, int P, int N>
__device__ __forceinline__ void row_stats(Team<TEAM>& team, const float (&v)[P][N], int lane, int d,
                                          int kind, float eps, float& mu, float& rho) {
  mu = 0.0f;
  if (kind == MONARCH_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < N; ++i) s += v[p][i];
    mu = team.sum(s) / static_cast<float>(d);
  }
  float s = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float c = (p * TEAM + lane) * N + i < d ? v[p][i] - mu : 0.0f;
      s = fmaf(c, c, s);
    }
  rho = 1.0f / sqrtf(team.sum(s) / static_cast<float>(d) + eps);
}

template <typename T, int TEAM, int P>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void sandwich_fwd_kernel(SandwichFwd a) {
  constexpr int N = PieceOf<T>::N, TEAMS = TEAM > 256 ? 1 : 256 / TEAM;
  __shared__ typename Team<TEAM>::Lds lds;
  Team<TEAM> team(&lds);
  const int lane = threadIdx.x % TEAM;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TEAM; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * TEAMS) {
    const int64_t off = row * a.d;
    const T* h = static_cast<const T*>(a.h) + off;
    u32x4 hr[P], yr[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      hr[p] = load_piece<T>(h, (p * TEAM + lane) * N, a.d);
      if (a.y)
        yr[p] = load_piece<T>(static_cast<const T*>(a.y) + off, (p * TEAM + lane) * N, a.d);
    }
    float v[P][N];
    f32x4 st = {0.0f, 1.0f, 0.0f, 1.0f};
    if (a.y) {
#pragma unroll
      for (int p = 0; p < P; ++p) PieceOf<T>::unpack(yr[p], v[p]);
      float mu = 0.0f, rho = 1.0f;
      if (a.post != MONARCH_NORM_NONE)
        row_stats<TEAM, P, N>(team, v, lane, a.d, a.post, a.eps, mu, rho);
      st[0] = mu, st[1] = rho;
      const int64_t goff = a.gate ? row / a.rows_per_gate * a.d : 0;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N;
        float w[N], b[N], g[N], hv[N];
        load_or<T, N>(a.post_w, 0, at, a.d, 1.0f, w);
        load_or<T, N>(a.post_b, 0, at, a.d, 0.0f, b);
        load_or<T, N>(a.gate, goff, at, a.d, 1.0f, g);
        PieceOf<T>::unpack(hr[p], hv);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float u = fmaf((v[p][i] - mu) * rho, w[i], b[i]);
          v[p][i] = fmaf(a.skip, hv[i], a.branch * g[i] * u);
          if (at + i >= a.d) v[p][i] = 0.0f;
        }
        if (at < a.d)
          store_piece<T>(static_cast<T*>(a.h_out) + off, at, a.d, PieceOf<T>::pack(v[p]));
      }
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) PieceOf<T>::unpack(hr[p], v[p]);
    }
    if (a.pre != MONARCH_NORM_NONE) {
      float mu, rho;
      row_stats<TEAM, P, N>(team, v, lane, a.d, a.pre, a.eps, mu, rho);
      st[2] = mu, st[3] = rho;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N;
        if (at < a.d) {
          float w[N], b[N], n[N];
          load_or<T, N>(a.pre_w, 0, at, a.d, 1.0f, w);
          load_or<T, N>(a.pre_b, 0, at, a.d, 0.0f, b);
#pragma unroll
          for (int i = 0; i < N; ++i) n[i] = fmaf((v[p][i] - mu) * rho, w[i], b[i]);
          store_piece<T>(static_cast<T*>(a.n_out) + off, at, a.d, PieceOf<T>::pack(n));
        }
      }
    }
    if (lane == 0) *reinterpret_cast<f32x4*>(a.stats + row * 4) = st;
  }
}

// ------------------------------------------------------------------ backward

// How the rows of a backward call are cut. CHUNK: chunk c holds rows of one
// gate row only (chunk / cpg), and its sums are of D alone; the gate and the
// branch scale are applied when the chunks are joined. UNIT: many short gate
// runs (down to one row each); each is summed by one team, which stores its
// dgate row itself, and the chunk's sums are of g * D.
struct SandwichBwd {
  const void *dh_out, *dn, *h_out, *y;
  const float* stats;
  const void *post_w, *post_b, *gate, *pre_w, *pre_b;
  void *dh, *dy, *dgate;
  float* part;          // [chunks][sums][d]
  int64_t rows, rows_per_gate, chunk_rows, cpg;
  int d, post, pre, sums;
  int s_post, s_postb, s_pre, s_preb;   // index of each sum in a chunk, -1: not taken
  float skip, branch;
};

template <typename T, int TEAM, int P, bool UNIT, bool BIAS>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void sandwich_bwd_kernel(SandwichBwd a) {
  constexpr int N = PieceOf<T>::N, WG = TEAM > 256 ? TEAM : 256, TEAMS = WG / TEAM;
  constexpr int COLS = TEAM * P * N;
  __shared__ typename Team<TEAM>::Lds lds;
  __shared__ float join[TEAMS > 1 ? TEAMS * COLS : 1];
  Team<TEAM> team(&lds);
  const int lane = threadIdx.x % TEAM, tm = threadIdx.x / TEAM;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  // rows [first, last) of this team, taken every `step`
  int64_t first, last;
  int step;
  int64_t group = 0;
  if constexpr (UNIT) {
    // chunk_rows counts whole gate runs here: this team's own range of them
    const int64_t units = a.rows / a.rows_per_gate;
    const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * TEAMS + tm) * a.chunk_rows;
    const int64_t u1 = u0 + a.chunk_rows < units ? u0 + a.chunk_rows : units;
    first = u0 * a.rows_per_gate;
    last = u1 * a.rows_per_gate;
    step = 1;
  } else {
    group = blockIdx.x / a.cpg;
    const int64_t c = blockIdx.x - group * a.cpg;
    const int64_t end = (group + 1) * a.rows_per_gate;
    first = group * a.rows_per_gate + c * a.chunk_rows;
    last = first + a.chunk_rows < end ? first + a.chunk_rows : end;
    first += tm;
    step = TEAMS;
  }
  float post_w[P][N], pre_w[P][N], gate[P][N], post_b[BIAS ? P : 1][N];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int at = (p * TEAM + lane) * N;
    load_or<T, N>(a.post_w, 0, at, a.d, 1.0f, post_w[p]);
    load_or<T, N>(a.pre_w, 0, at, a.d, 1.0f, pre_w[p]);
    if constexpr (BIAS) load_or<T, N>(a.post_b, 0, at, a.d, 0.0f, post_b[p]);
    if constexpr (!UNIT) load_or<T, N>(a.gate, group * a.d, at, a.d, 1.0f, gate[p]);
  }
  float s_post[P][N] = {}, s_pre[P][N] = {}, s_gate[UNIT ? P : 1][N] = {};
  float s_postb[BIAS ? P : 1][N] = {}, s_preb[BIAS ? P : 1][N] = {};
  int64_t left = a.rows_per_gate;   // UNIT: rows of the gate run still to come
  for (int64_t row = first; row < last; row += step) {
    const int64_t off = row * a.d;
    const f32x4 st = *reinterpret_cast<const f32x4*>(a.stats + row * 4);
    u32x4 dhr[P], dnr[P], hr[P], yr[P], gr[UNIT ? P : 1];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = (p * TEAM + lane) * N;
      const u32x4 zero = {0, 0, 0, 0};
      dhr[p] = dnr[p] = hr[p] = yr[p] = zero;
      if (a.pre != MONARCH_NORM_NONE) {
        dnr[p] = load_piece<T>(static_cast<const T*>(a.dn) + off, at, a.d);
        hr[p] = load_piece<T>(static_cast<const T*>(a.h_out) + off, at, a.d);
      }
      if (a.dh_out) dhr[p] = load_piece<T>(static_cast<const T*>(a.dh_out) + off, at, a.d);
      if (a.y) yr[p] = load_piece<T>(static_cast<const T*>(a.y) + off, at, a.d);
      if constexpr (UNIT)
        gr[p] = load_piece<T>(static_cast<const T*>(a.gate) + row / a.rows_per_gate * a.d, at, a.d);
    }
    float D[P][N];
#pragma unroll
    for (int p = 0; p < P; ++p) PieceOf<T>::unpack(dhr[p], D[p]);
    if (a.pre != MONARCH_NORM_NONE) {
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float dn[N], h[N];
        PieceOf<T>::unpack(dnr[p], dn);
        PieceOf<T>::unpack(hr[p], h);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float hat = (h[i] - st[2]) * st[3], q = dn[i] * pre_w[p][i];
          s[0] = fmaf(q, hat, s[0]);
          s[1] += q;
          s_pre[p][i] = fmaf(dn[i], hat, s_pre[p][i]);
          if constexpr (BIAS) s_preb[p][i] += dn[i];
        }
      }
      team.template reduce<SumOp, 2>(s);
      const float c1 = s[0] * inv_d, c2 = a.pre == MONARCH_NORM_LAYER ? s[1] * inv_d : 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float dn[N], h[N];
        PieceOf<T>::unpack(dnr[p], dn);
        PieceOf<T>::unpack(hr[p], h);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float hat = (h[i] - st[2]) * st[3], q = dn[i] * pre_w[p][i];
          D[p][i] = fmaf(st[3], q - fmaf(hat, c1, c2), D[p][i]);
        }
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = (p * TEAM + lane) * N;
      if (at < a.d) {
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = a.skip * D[p][i];
        store_piece<T>(static_cast<T*>(a.dh) + off, at, a.d, PieceOf<T>::pack(o));
      }
    }
    if (a.y) {
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float y[N], g[N];
        PieceOf<T>::unpack(yr[p], y);
        if constexpr (UNIT) PieceOf<T>::unpack(gr[p], g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float hat = (y[i] - st[0]) * st[1];
          const float gv = UNIT ? g[i] : gate[p][i];
          const float q2 = a.branch * gv * D[p][i] * post_w[p][i];
          s[0] = fmaf(q2, hat, s[0]);
          s[1] += q2;
          if constexpr (UNIT) {
            const float u = BIAS ? fmaf(hat, post_w[p][i], post_b[p][i]) : hat * post_w[p][i];
            s_gate[p][i] = fmaf(D[p][i], u, s_gate[p][i]);
            s_post[p][i] = fmaf(gv * D[p][i], hat, s_post[p][i]);
            if constexpr (BIAS) s_postb[p][i] = fmaf(gv, D[p][i], s_postb[p][i]);
          } else {
            s_post[p][i] = fmaf(D[p][i], hat, s_post[p][i]);
            if constexpr (BIAS) s_postb[p][i] += D[p][i];
          }
        }
      }
      float c1 = 0.0f, c2 = 0.0f;
      if (a.post != MONARCH_NORM_NONE) {
        team.template reduce<SumOp, 2>(s);
        c1 = s[0] * inv_d;
        c2 = a.post == MONARCH_NORM_LAYER ? s[1] * inv_d : 0.0f;
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N;
        float y[N], g[N], o[N];
        PieceOf<T>::unpack(yr[p], y);
        if constexpr (UNIT) PieceOf<T>::unpack(gr[p], g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float hat = (y[i] - st[0]) * st[1];
          const float gv = UNIT ? g[i] : gate[p][i];
          o[i] = st[1] * (a.branch * gv * D[p][i] * post_w[p][i] - fmaf(hat, c1, c2));
        }
        if (at < a.d) store_piece<T>(static_cast<T*>(a.dy) + off, at, a.d, PieceOf<T>::pack(o));
      }
    }
    if constexpr (UNIT) {
      if (--left == 0) {
        left = a.rows_per_gate;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int at = (p * TEAM + lane) * N;
          float o[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            o[i] = a.branch * s_gate[p][i];
            s_gate[p][i] = 0.0f;
          }
          if (a.dgate && at < a.d)
            store_piece<T>(static_cast<T*>(a.dgate) + row / a.rows_per_gate * a.d, at, a.d,
                           PieceOf<T>::pack(o));
        }
      }
    }
  }
  // this chunk's sums: the teams' are added in team order
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.sums * a.d;
  auto put = [&](int which, const float(&s)[P][N]) {
    if (which < 0) return;
    float* out = part + static_cast<int64_t>(which) * a.d;
    if constexpr (TEAMS == 1) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int at = (p * TEAM + lane) * N + i;
          if (at < a.d) out[at] = s[p][i];
        }
    } else {
      __syncthreads();
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) join[tm * COLS + (p * TEAM + lane) * N + i] = s[p][i];
      __syncthreads();
      for (int at = threadIdx.x; at < a.d; at += WG) {
        float t = join[at];
#pragma unroll
        for (int k = 1; k < TEAMS; ++k) t += join[k * COLS + at];
        out[at] = t;
      }
    }
  };
  put(a.s_post, s_post);
  put(a.s_pre, s_pre);
  if constexpr (BIAS) {
    put(a.s_postb, s_postb);
    put(a.s_preb, s_preb);
  }
}

// Joins the chunks' sums. A job is one output row: the weight gradients (sums
// over every chunk, weighted by the chunk's gate row) and, when chunks hold
// sums of D alone, one dgate row each. A workgroup takes 64 columns; 16 slices
// of 64 threads sum contiguous chunk ranges, and the slices are added in order.
struct SandwichJoin {
  const float* part;
  const void *gate, *post_w, *post_b;   // gate: null where the sums hold it already
  void *dgate, *dpost_w, *dpost_b, *dpre_w, *dpre_b;
  int64_t chunks, cpg;
  int d, sums, s_post, s_postb, s_pre, s_preb;
  float branch;
};

constexpr int JC = 64, JS = 16;
constexpr int kWeightJobs = 4;   // post_w, post_b, pre_w, pre_b; then one job a gate row

template <typename T>
__global__ __launch_bounds__(JC* JS) void sandwich_join_kernel(SandwichJoin a) {
  __shared__ float buf[2][JS][JC];
  const int col = threadIdx.x % JC, slice = threadIdx.x / JC;
  const int at = blockIdx.y * JC + col;
  const int64_t job = blockIdx.x;
  int which, which2 = -1;
  int64_t c0 = 0, c1 = a.chunks;
  bool gated = false;
  void* out;
  if (job < kWeightJobs) {
    which = job == 0 ? a.s_post : job == 1 ? a.s_postb : job == 2 ? a.s_pre : a.s_preb;
    out = job == 0 ? a.dpost_w : job == 1 ? a.dpost_b : job == 2 ? a.dpre_w : a.dpre_b;
    gated = job < 2 && a.gate;
  } else {
    which = a.s_post;
    which2 = a.post_b ? a.s_postb : -1;
    c0 = (job - kWeightJobs) * a.cpg;
    c1 = c0 + a.cpg;
    out = static_cast<T*>(a.dgate) + (job - kWeightJobs) * a.d;
  }
  if (!out || which < 0) return;   // the whole workgroup
  const int64_t per = (c1 - c0 + JS - 1) / JS;
  const int64_t b = c0 + slice * per, e = b + per < c1 ? b + per : c1;
  float s = 0.0f, s2 = 0.0f;
  if (at < a.d) {
    const float* p = a.part + static_cast<int64_t>(which) * a.d + at;
    const float* p2 = a.part + static_cast<int64_t>(which2 < 0 ? 0 : which2) * a.d + at;
    const int64_t stride = static_cast<int64_t>(a.sums) * a.d;
#pragma unroll 4
    for (int64_t c = b; c < e; ++c) {
      float v = p[c * stride];
      if (gated) v *= Io<T>::load(a.gate, c / a.cpg * a.d + at);
      s += v;
      if (which2 >= 0) s2 += p2[c * stride];
    }
  }
  buf[0][slice][col] = s;
  buf[1][slice][col] = s2;
  __syncthreads();
  if (slice || at >= a.d) return;
#pragma unroll
  for (int k = 1; k < JS; ++k) {
    s += buf[0][k][col];
    s2 += buf[1][k][col];
  }
  if (job >= kWeightJobs) {
    s *= a.post_w ? Io<T>::load(a.post_w, at) : 1.0f;
    if (which2 >= 0) s = fmaf(s2, Io<T>::load(a.post_b, at), s);
  }
  if (job < 2 || job >= kWeightJobs) s *= a.branch;
  if constexpr (sizeof(T) == 2)
    static_cast<uint16_t*>(out)[at] = f32_to_bf16(s);
  else
    static_cast<float*>(out)[at] = s;
}

// ---------------------------------------------------------------- host side

struct Shape {
  int team, pieces;
};

// The smallest team (of at least `least` threads) whose threads hold at most
// `most` pieces of a row.
Shape shape_of(int64_t d, bool bf16, int least, int most) {
  const int n = bf16 ? 8 : 4;
  const int64_t pieces = (d + n - 1) / n;
  static const int teams[] = {16, 32, 64, 256, 1024};
  for (int t : teams)
    if (t >= least && (pieces + t - 1) / t <= most)
      return {t, static_cast<int>((pieces + t - 1) / t)};
  return {1024, static_cast<int>((pieces + 1023) / 1024)};
}

struct BwdPlan {
  Shape shape;
  bool unit, bias;
  int64_t chunks, chunk_rows, cpg, rows_per_gate;
  int sums, s_post, s_postb, s_pre, s_preb;
  size_t ws;
};

constexpr int64_t kChunks = 512;      // workgroups aimed at: two a CU
constexpr int64_t kUnitRows = 32;     // gate runs up to this long are a team's own

// Everything about a backward call that depends on sizes alone (`with`: which
// of post_w, post_b, gate, pre_w, pre_b there are, as the sums they need).
BwdPlan bwd_plan(int64_t rows, int64_t d, int64_t gates, bool has_y, bool post_bias, bool has_pre,
                 bool pre_bias, bool bf16) {
  BwdPlan p = {};
  p.shape = shape_of(d, bf16, 32, bf16 ? 3 : 4);
  p.bias = post_bias || pre_bias;
  p.rows_per_gate = gates > 0 ? rows / gates : rows;
  p.unit = rows > 0 && gates > 1 && p.rows_per_gate <= kUnitRows;
  const int teams = p.shape.team >= 256 ? 1 : 256 / p.shape.team;
  if (rows == 0) {
    p.cpg = 0;   // no chunk: every sum is empty
  } else if (p.unit) {
    const int64_t units = gates, slots = kChunks * teams;
    p.chunk_rows = (units + slots - 1) / slots;
    p.chunks = (units + p.chunk_rows * teams - 1) / (p.chunk_rows * teams);
    p.cpg = 1;
  } else {
    const int64_t g = gates > 0 ? gates : 1;
    int64_t cpg = (kChunks + g - 1) / g;
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
  if (rows < 0 || rows >= kLimit || d <= 0 || d > kMaxFeatures || gates < 0) return MONARCH_ERR_SHAPE;
  if (gates > 0 && (rows % gates != 0 || (rows > 0 && gates > rows))) return MONARCH_ERR_SHAPE;
  return MONARCH_OK;
}

template <typename T, int TEAM, int P>
void fwd_launch(const SandwichFwd& a, hipStream_t s) {
  constexpr int WG = TEAM > 256 ? TEAM : 256, TEAMS = WG / TEAM;
  int64_t grid = (a.rows + TEAMS - 1) / TEAMS;
  if (grid > (1 << 20)) grid = 1 << 20;   // fewer than 2^32 threads; the rest by stride
  hipLaunchKernelGGL((sandwich_fwd_kernel<T, TEAM, P>), dim3(static_cast<unsigned>(grid)), dim3(WG),
                     0, s, a);
}

template <typename T, int TEAM, int P>
void bwd_launch(const SandwichBwd& a, const BwdPlan& p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.chunks)), block(TEAM > 256 ? TEAM : 256);
  if (p.unit && p.bias)
    hipLaunchKernelGGL((sandwich_bwd_kernel<T, TEAM, P, true, true>), grid, block, 0, s, a);
  else if (p.unit)
    hipLaunchKernelGGL((sandwich_bwd_kernel<T, TEAM, P, true, false>), grid, block, 0, s, a);
  else if (p.bias)
    hipLaunchKernelGGL((sandwich_bwd_kernel<T, TEAM, P, false, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((sandwich_bwd_kernel<T, TEAM, P, false, false>), grid, block, 0, s, a);
}

#define MONARCH_TEAM_CASE(CALL, T, TEAM, P) \
  case (TEAM) * 8 + (P):                    \
    CALL(T, TEAM, P);                       \
    break;

hipError_t launch_fwd(const SandwichFwd& a, bool bf16, hipStream_t s) {
  const Shape sh = shape_of(a.d, bf16, 16, 4);
#define FWD(T, TEAM, P) fwd_launch<T, TEAM, P>(a, s)
#define FWD4(T, TEAM)                \
  MONARCH_TEAM_CASE(FWD, T, TEAM, 1) \
  MONARCH_TEAM_CASE(FWD, T, TEAM, 2) \
  MONARCH_TEAM_CASE(FWD, T, TEAM, 3) \
  MONARCH_TEAM_CASE(FWD, T, TEAM, 4)
  if (bf16) {
    switch (sh.team * 8 + sh.pieces) {
      FWD4(uint16_t, 16)
      FWD4(uint16_t, 32)
      FWD4(uint16_t, 64)
      FWD4(uint16_t, 256)
      MONARCH_TEAM_CASE(FWD, uint16_t, 1024, 2)
      default: return hipErrorInvalidConfiguration;
    }
  } else {
    switch (sh.team * 8 + sh.pieces) {
      FWD4(float, 16)
      FWD4(float, 32)
      FWD4(float, 64)
      FWD4(float, 256)
      MONARCH_TEAM_CASE(FWD, float, 1024, 2)
      MONARCH_TEAM_CASE(FWD, float, 1024, 3)
      MONARCH_TEAM_CASE(FWD, float, 1024, 4)
      default: return hipErrorInvalidConfiguration;
    }
  }
#undef FWD4
#undef FWD
  return hipGetLastError();
}

hipError_t launch_bwd(const SandwichBwd& a, const BwdPlan& p, bool bf16, hipStream_t s) {
#define BWD(T, TEAM, P) bwd_launch<T, TEAM, P>(a, p, s)
#define BWD3(T, TEAM)                \
  MONARCH_TEAM_CASE(BWD, T, TEAM, 1) \
  MONARCH_TEAM_CASE(BWD, T, TEAM, 2) \
  MONARCH_TEAM_CASE(BWD, T, TEAM, 3)
  if (bf16) {
    switch (p.shape.team * 8 + p.shape.pieces) {
      BWD3(uint16_t, 32)
      BWD3(uint16_t, 64)
      BWD3(uint16_t, 256)
      MONARCH_TEAM_CASE(BWD, uint16_t, 1024, 1)
      MONARCH_TEAM_CASE(BWD, uint16_t, 1024, 2)
      default: return hipErrorInvalidConfiguration;
    }
  } else {
    switch (p.shape.team * 8 + p.shape.pieces) {
      BWD3(float, 32)
      MONARCH_TEAM_CASE(BWD, float, 32, 4)
      BWD3(float, 64)
      MONARCH_TEAM_CASE(BWD, float, 64, 4)
      BWD3(float, 256)
      MONARCH_TEAM_CASE(BWD, float, 256, 4)
      MONARCH_TEAM_CASE(BWD, float, 1024, 2)
      MONARCH_TEAM_CASE(BWD, float, 1024, 3)
      MONARCH_TEAM_CASE(BWD, float, 1024, 4)
      default: return hipErrorInvalidConfiguration;
    }
  }
#undef BWD3
#undef BWD
  return hipGetLastError();
}
#undef MONARCH_TEAM_CASE

hipError_t launch_join(const SandwichJoin& a, int64_t jobs, bool bf16, hipStream_t s) {
  // jobs < 2^21 at 1024 threads stay below 2^32 threads a launch: gate rows
  // summed here have more than kUnitRows rows each, columns are at most 16384
  const dim3 grid(static_cast<unsigned>(jobs), static_cast<unsigned>((a.d + JC - 1) / JC));
  if (bf16)
    hipLaunchKernelGGL((sandwich_join_kernel<uint16_t>), grid, dim3(JC * JS), 0, s, a);
  else
    hipLaunchKernelGGL((sandwich_join_kernel<float>), grid, dim3(JC * JS), 0, s, a);
  return hipGetLastError();
}

bool any_misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (misaligned(p)) return true;
  return false;
}

}  // namespace
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
  a.rows = rows, a.rows_per_gate = gates > 0 ? rows / gates : rows;
  a.d = static_cast<int>(features), a.post = post_norm, a.pre = pre_norm;
  a.skip = skip_scale, a.branch = branch_scale, a.eps = eps;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Tracer tr{events, n_events, 0, s};
  st = record_hip(tr.mark());
  if (st) return st;
  st = record_hip(launch_fwd(a, dtype == MONARCH_BF16, s));
  if (st) return st;
  return record_hip(tr.mark());
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
      (dpre_w && !pre_w) || (dpre_b && !pre_b))
    return MONARCH_ERR_NULL;
  const BwdPlan p = bwd_plan(rows, features, gates, y || rows == 0, post_b != nullptr, has_pre,
                             pre_b != nullptr, bf16);
  if (rows > 0 && p.ws > 0 && !workspace) return MONARCH_ERR_NULL;
  if (rows > 0 && workspace_bytes < p.ws) return MONARCH_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Tracer tr{events, n_events, 0, s};
  if (rows > 0) {
    SandwichBwd a;
    a.dh_out = dh_out, a.dn = dn, a.h_out = h_out, a.y = y;
    a.stats = static_cast<const float*>(stats);
    a.post_w = post_w, a.post_b = post_b, a.gate = gates > 0 ? gate : nullptr;
    a.pre_w = has_pre ? pre_w : nullptr, a.pre_b = has_pre ? pre_b : nullptr;
    a.dh = dh, a.dy = dy, a.dgate = dgate, a.part = static_cast<float*>(workspace);
    a.rows = rows, a.rows_per_gate = p.rows_per_gate, a.chunk_rows = p.chunk_rows, a.cpg = p.cpg;
    a.d = static_cast<int>(features), a.post = post_norm, a.pre = pre_norm, a.sums = p.sums;
    a.s_post = p.s_post, a.s_postb = p.s_postb, a.s_pre = p.s_pre, a.s_preb = p.s_preb;
    a.skip = skip_scale, a.branch = branch_scale;
    st = record_hip(tr.mark());
    if (st) return st;
    st = record_hip(launch_bwd(a, p, bf16, s));
    if (st) return st;
  }
  if (dpost_w || dpost_b || dgate || dpre_w || dpre_b) {
    SandwichJoin j;
    j.part = static_cast<const float*>(workspace);
    j.gate = gates > 0 && !p.unit ? gate : nullptr;
    j.post_w = post_w, j.post_b = post_b;
    j.dgate = dgate, j.dpost_w = dpost_w, j.dpost_b = dpost_b, j.dpre_w = dpre_w, j.dpre_b = dpre_b;
    j.chunks = p.chunks, j.cpg = p.cpg;
    j.d = static_cast<int>(features), j.sums = p.sums;
    j.s_post = p.s_post, j.s_postb = p.s_postb, j.s_pre = p.s_pre, j.s_preb = p.s_preb;
    j.branch = branch_scale;
    const int64_t jobs = kWeightJobs + (dgate && !p.unit ? gates : 0);
    st = record_hip(tr.mark());
    if (st) return st;
    st = record_hip(launch_join(j, jobs, bf16, s));
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
