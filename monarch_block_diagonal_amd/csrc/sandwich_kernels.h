// Sandwich norm, the kernels: the norm after a block, its gate, the scaled residual
// join and the norm before the next block, forward and backward.
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
// read once and written once, which is what bounds both passes (about 10
// operations a value forward, 35 backward). All arithmetic and all sums are
// fp32; results are rounded once, at their store. n is computed from h' before
// its rounding, and the backward pass needs that h' too: in bf16 the forward pass keeps 4
// more bits a value beside the statistics (low_bits). From h_out alone dw_pre was 2.6e-3
// off the formula's where one rounding is 1.7e-3, and more where a LAYER row's mean is
// larger than its spread. The half byte a value is 6% of the forward pass's bytes and 4%
// of the backward pass's (forward / backward and join, 16384 x 768 18.2 / 31.7 us
// without it, 19.7 / 35.0 with; 8192 x 16384 with a gate a row 248 / 428 and 264 / 440).
#pragma once

#include <type_traits>

#include "monarch.h"
#include "sandwich.h"
#include "team.h"

namespace monarch {
namespace {

// A piece of an optional row (weights, biases, a gate row): without one, ones or
// zeros, so that the arithmetic is the same.
template <typename T, Rows R>
__device__ __forceinline__ u32x4 par_piece(const void* p, int64_t off, int at, int d, float fill) {
  if (p) return load_piece<T, R>(static_cast<const T*>(p) + off, at, d);
  const uint32_t w = sizeof(T) == 2 ? (__float_as_uint(fill) >> 16) * 0x10001u : __float_as_uint(fill);
  return u32x4{w, w, w, w};
}

// Four more bits of each of a piece's values than their roundings to bf16 hold: the
// difference from the rounding in sixteenths of its last place, -8 .. 7. A value that
// bf16 holds gives 0; what is left is at most a sixteenth, mostly a 32nd, of a last place.
// The difference is that of the bit patterns, which also runs over exponents: the
// pattern's low half as a signed number, one less where the upper half is even, so that
// a tie (to even) falls on its side. Two values at a time in 16-bit halves; element 2 k
// in bits 4 k, element 2 k + 1 in bits 16 + 4 k.
__device__ __forceinline__ uint32_t low_bits(const float (&v)[8]) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  uint32_t word = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = __float_as_uint(v[2 * k]), b = __float_as_uint(v[2 * k + 1]);
    const uint32_t low = __builtin_amdgcn_perm(b, a, 0x05040100u);
    const uint32_t even = ~__builtin_amdgcn_perm(b, a, 0x07060302u) & 0x00010001u;
    s16x2 x, one, t = {0x800, 0x800};
    __builtin_memcpy(&x, &low, 4);
    __builtin_memcpy(&one, &even, 4);
    t = __builtin_elementwise_add_sat(static_cast<s16x2>(x - one), t);
    uint32_t top;   // four bits at the top of each half
    __builtin_memcpy(&top, &t, 4);
    word = (word >> 4 & 0x0fff0fffu) | (top & 0xf000f000u);
  }
  return word;
}

// A piece of h' for the backward pass: h_out with the bits that were kept.
template <typename T, int N>
__device__ __forceinline__ void unpack_low(const u32x4& r, uint32_t word, float (&v)[N]) {
  PieceOf<T>::unpack(r, v);
  if constexpr (N == 8)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int q = static_cast<int>(word << (28 - 4 * (i / 2) - 16 * (i % 2))) >> 28;
      v[i] = __uint_as_float(__float_as_uint(v[i]) + (static_cast<uint32_t>(q) << 12));
    }
}

// mean and 1/sqrt(mean square about it + eps) of the team's row (zero past d)
template <Rows R, int TEAM, int P, int N>
__device__ __forceinline__ void row_stats(Team<TEAM>& team, const float (&v)[P][N], int lane, int d,
                                          int kind, float eps, float& mu, float& rho) {
  mu = 0.0f;
  float q = 0.0f;
  if (kind == MONARCH_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < N; ++i) s += v[p][i];
    mu = team.sum(s) / static_cast<float>(d);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float c[N];
#pragma unroll
      for (int i = 0; i < N; ++i) c[i] = v[p][i] - mu;
      mask<R, N>(c, (p * TEAM + lane) * N, d);
#pragma unroll
      for (int i = 0; i < N; ++i) q = fmaf(c[i], c[i], q);
    }
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < N; ++i) q = fmaf(v[p][i], v[p][i], q);
  }
  rho = 1.0f / sqrtf(team.sum(q) / static_cast<float>(d) + eps);
}

// The start of a row. Where a row is the workgroup's it is held in scalar registers
// and taken as it is: the compiler would keep the sum of the tensor's address and each
// piece's place over the loop instead, two registers a piece and tensor (2048 x 16384
// fp32 backward and join 206 -> 176 us).
template <int TEAM, typename T, typename V>
__device__ __forceinline__ auto row_start(V* p, int64_t off) {
  typedef typename std::conditional<std::is_const<V>::value, const T, T>::type E;
  E* r = static_cast<E*>(p) + off;
  if constexpr (TEAM > 64) asm volatile("" : "+s"(r));
  return r;
}

// One row a team. A team of 1024 threads leaves room for one workgroup a CU: it
// takes rows in turn and loads the next one while the present one is normed a
// second time. Measured (every tensor once): 16384 x 768 bf16 19.7 us, 5.4 TB/s; 10000 x
// 625 fp32 20.3 us, 4.9 TB/s; 8192 x 16384 bf16 with a gate a row 264 us, 5.3 TB/s, where a
// copy of that size reaches 5.6; one row of 768 4.1 us, the launch. Small teams of 32 lanes x 3 pieces beat 64 x 2 for 768 features (20.3
// against 21.1 us): every lane holds whole pieces.
template <typename T, int TEAM, int P, bool BIAS, Rows R>
__global__ __launch_bounds__(TEAM > 64 ? TEAM : 256, TEAM > 512 || R == WHOLE ? 4 : 3) void sandwich_fwd_kernel(SandwichFwd a) {
  constexpr int N = PieceOf<T>::N, TEAMS = TEAM > 64 ? 1 : 256 / TEAM;
  constexpr bool AHEAD = TEAM == 1024 && P <= 3;
  __shared__ typename Team<TEAM>::Lds lds;
  Team<TEAM> team(&lds);
  const int lane = TEAMS == 1 ? threadIdx.x : threadIdx.x % TEAM, tm = TEAMS == 1 ? 0 : threadIdx.x / TEAM;
  const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
  u32x4 hr[P], yr[P];
  auto load = [&](int64_t row) {
    const int d = anew(a.d);
    const T *h = row_start<TEAM, T>(a.h, row * d), *y = row_start<TEAM, T>(a.y, row * d);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = (p * TEAM + lane) * N;
      hr[p] = load_piece<T, R>(h, at, d);
      if (a.y) yr[p] = load_piece<T, R>(y, at, d);
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + tm;
  if (AHEAD && row < a.rows) load(row);
  for (; row < a.rows; row += step) {
    const int d = anew(a.d);
    const int64_t off = row * d;
    if constexpr (!AHEAD) load(row);
    float v[P][N];
    float mu_y = 0.0f, rho_y = 1.0f, mu_h = 0.0f, rho_h = 1.0f;
    if (a.y) {
      if (a.post != MONARCH_NORM_NONE) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          PieceOf<T>::unpack(yr[p], v[p]);
          if constexpr (R != WHOLE) mask<R, N>(v[p], (p * TEAM + lane) * N, d);
        }
        row_stats<R, TEAM, P, N>(team, v, lane, d, a.post, a.eps, mu_y, rho_y);
      }
      const int64_t goff = a.gate ? row / a.rows_per_gate * d : 0;
      // branch * yhat, so that the scale costs nothing a value
      const float scale = a.branch * rho_y, mean = mu_y * scale;
      T* h_out = row_start<TEAM, T>(a.h_out, off);
      uint32_t* low = row_start<TEAM, uint32_t>(a.low, row * ((d + N - 1) / N));
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N;
        float w[N], b[N], g[N], t[N];
        forget(yr[p]);
        PieceOf<T>::unpack(yr[p], v[p]);
        PieceOf<T>::unpack(par_piece<T, R>(a.post_w, 0, at, d, 1.0f), w);
        if constexpr (BIAS)
          PieceOf<T>::unpack(par_piece<T, R>(a.post_b, 0, at, d, 0.0f), b);
        PieceOf<T>::unpack(par_piece<T, R>(a.gate, goff, at, d, 1.0f), g);
        PieceOf<T>::unpack(hr[p], t);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float u = fmaf(v[p][i], scale, -mean) * w[i];
          if constexpr (BIAS) u = fmaf(a.branch, b[i], u);
          v[p][i] = fmaf(a.skip, t[i], g[i] * u);
        }
        store_piece<T, R>(h_out, at, d, PieceOf<T>::pack(v[p]));
        if constexpr (N == 8)
          if (a.low && at < d)
            __builtin_nontemporal_store(low_bits(v[p]), low + static_cast<unsigned>(at) / 8);
        mask<R, N>(v[p], at, d);
      }
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        PieceOf<T>::unpack(hr[p], v[p]);
        if constexpr (R != WHOLE) mask<R, N>(v[p], (p * TEAM + lane) * N, d);
      }
    }
    if (AHEAD && row + step < a.rows) load(row + step);
    if (a.pre != MONARCH_NORM_NONE) {
      row_stats<R, TEAM, P, N>(team, v, lane, d, a.pre, a.eps, mu_h, rho_h);
      const float mean_h = mu_h * rho_h;
      T* n_out = row_start<TEAM, T>(a.n_out, off);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N;
        float w[N], b[N];
        PieceOf<T>::unpack(par_piece<T, R>(a.pre_w, 0, at, d, 1.0f), w);
        if constexpr (BIAS)
          PieceOf<T>::unpack(par_piece<T, R>(a.pre_b, 0, at, d, 0.0f), b);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          v[p][i] = fmaf(v[p][i], rho_h, -mean_h) * w[i];
          if constexpr (BIAS) v[p][i] += b[i];
        }
        store_piece<T, R>(n_out, at, d, PieceOf<T>::pack(v[p]));
      }
    }
    if (lane == 0) *reinterpret_cast<f32x4*>(a.stats + row * 4) = f32x4{mu_y, rho_y, mu_h, rho_h};
  }
}

// A thread's sums over rows for its own columns: in registers, or in LDS (WG
// threads side by side, 16 bytes each), where they would not leave registers for
// the row itself.
template <int WG, int P, int N, bool IN_LDS>
struct Sums {
  float v[IN_LDS ? 1 : P][N];
  f32x4* lds;
  __device__ __forceinline__ void clear(f32x4* l) {
    lds = l;
    if constexpr (IN_LDS) {
#pragma unroll
      for (int k = 0; k < P * N / 4; ++k) lds[k * WG + threadIdx.x] = f32x4{0, 0, 0, 0};
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) v[p][i] = 0.0f;
    }
  }
  // adds x[i] to the sums of piece p
  __device__ __forceinline__ void add(int p, const float (&x)[N]) {
    if constexpr (IN_LDS) {
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        f32x4& s = lds[(p * (N / 4) + k) * WG + threadIdx.x];
        f32x4 t = s;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] += x[4 * k + i];
        s = t;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[p][i] += x[i];
    }
  }
  // column i of piece p of a thread of the workgroup (LDS)
  __device__ __forceinline__ float at(int p, int i, int thread) const {
    return reinterpret_cast<const float*>(&lds[(p * (N / 4) + i / 4) * WG + thread])[i % 4];
  }
};

// Each team takes the rows of its chunk in turn and keeps its columns' sums over
// them, so that the parameters' gradients cost a partial row a chunk: two chunks
// a CU (three made the partial rows cost more than they hid: 30 -> 37 us for 16384
// x 768 bf16). Wide rows leave no registers for the sums: they lie in LDS (131 KB
// for 16384 columns; in registers the kernel spilled, 1208 -> 488 us), parameters
// are read again from the caches, and the next row's dn and h' are under way during
// the second half of a row. Measured: 16384 x 768 bf16 with 16 gates 31 us, 5.1
// TB/s; 10000 x 625 fp32 with biases 30.6 us, 4.9 TB/s; 8192 x 16384 bf16 with a gate a row 429
// us, 5.1 TB/s (calls among others; run apart, in a kernel trace, up to a tenth longer).
template <typename T, int TEAM, int P, int GATE, bool BIAS, Rows R>
__global__ __launch_bounds__(TEAM > 64 ? TEAM : 256) void sandwich_bwd_kernel(SandwichBwd a) {
  constexpr int N = PieceOf<T>::N, WG = TEAM > 64 ? TEAM : 256, TEAMS = WG / TEAM;
  constexpr int COLS = TEAM * P * N;
  // sums of post_w and pre_w in LDS (those of a cut row's long gate runs too: 16384 x
  // 767 bf16 37.6 -> 34.6 us, where short runs take 44.1 us in registers and 48.1 in
  // LDS); parameters read again for every row; the next row's first tensors loaded
  // ahead
  constexpr bool IN_LDS = TEAM > 64 || BIAS || (R == CUT && GATE == CHUNK);
  constexpr bool REREAD = TEAM > 256;
  constexpr bool LATE = TEAM > 512;   // 128 registers a thread: y's side is loaded last
  constexpr bool AHEAD = TEAM > 64 && !LATE;
  __shared__ typename Team<TEAM>::Lds lds;
  __shared__ f32x4 shared[IN_LDS ? 2 * WG * P * N / 4 : TEAMS > 1 ? TEAMS * COLS / 4 : 1];
  Team<TEAM> team(&lds);
  const int lane = TEAMS == 1 ? threadIdx.x : threadIdx.x % TEAM, tm = TEAMS == 1 ? 0 : threadIdx.x / TEAM;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  // rows [first, last) of this team, taken every `step`
  int64_t first, last, group = 0;
  int step = 1;
  if constexpr (GATE != CHUNK) {
    // chunk_rows counts whole gate runs here: this team's own range of them
    const int64_t units = a.rows / a.rows_per_gate;
    group = (static_cast<int64_t>(blockIdx.x) * TEAMS + tm) * a.chunk_rows;
    const int64_t u1 = group + a.chunk_rows < units ? group + a.chunk_rows : units;
    first = group * a.rows_per_gate;
    last = u1 * a.rows_per_gate;
  } else {
    group = blockIdx.x / a.cpg;
    const int64_t c = blockIdx.x - group * a.cpg;
    const int64_t end = (group + 1) * a.rows_per_gate;
    first = group * a.rows_per_gate + c * a.chunk_rows;
    last = first + a.chunk_rows < end ? first + a.chunk_rows : end;
    first += tm;
    step = TEAMS;
  }
  const u32x4 zero = {0, 0, 0, 0};
  u32x4 post_wr[P], pre_wr[P], gr[P];
  auto load_pre_pars = [&]() {
    const int d = anew(a.d);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = (p * TEAM + lane) * N;
      pre_wr[p] = par_piece<T, R>(a.pre_w, 0, at, d, 1.0f);
    }
  };
  auto load_post_pars = [&]() {
    const int d = anew(a.d);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = (p * TEAM + lane) * N;
      post_wr[p] = par_piece<T, R>(a.post_w, 0, at, d, 1.0f);
      if constexpr (GATE == CHUNK) {
        gr[p] = par_piece<T, R>(a.gate, group * d, at, d, 1.0f);
      }
    }
  };
  if constexpr (!REREAD) {
    load_pre_pars();
    load_post_pars();
  }
  Sums<WG, P, N, IN_LDS> s_post, s_pre;
  Sums<WG, BIAS ? P : 1, N, false> s_postb, s_preb;
  Sums<WG, GATE == RUN ? P : 1, N, false> s_gate;
  s_post.clear(shared);
  s_pre.clear(shared + (IN_LDS ? WG * P * N / 4 : 0));
  s_postb.clear(nullptr);
  s_preb.clear(nullptr);
  s_gate.clear(nullptr);
  int64_t left = a.rows_per_gate;   // RUN: rows of the gate run still to come

  u32x4 dnr[P], hr[P];
  uint32_t lowr[P];
  auto load_pre = [&](int64_t row) {
    const int d = anew(a.d);
    const T *dn = row_start<TEAM, T>(a.dn, row * d), *h = row_start<TEAM, T>(a.h_out, row * d);
    const uint32_t* low = row_start<TEAM, uint32_t>(a.low, row * a.low_row);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = (p * TEAM + lane) * N;
      dnr[p] = hr[p] = zero;
      // a word of another piece past the row, any where none are kept: both do not count
      // (low_word)
      lowr[p] = 0;
      if constexpr (N == 8) lowr[p] = low[at < d && a.low_row ? static_cast<unsigned>(at) / 8 : 0u];
      if (a.pre != MONARCH_NORM_NONE) {
        dnr[p] = load_piece<T, R>(dn, at, d);
        hr[p] = load_piece<T, R>(h, at, d);
      }
    }
  };
  auto low_word = [&](int p) {
    return (p * TEAM + lane) * N < a.d && a.low_row ? lowr[p] : 0u;
  };
  if (AHEAD && first < last) load_pre(first);
  for (int64_t row = first; row < last; row += step) {
    const int d = anew(a.d);
    const int64_t off = row * d;
    const f32x4 st = *reinterpret_cast<const f32x4*>(a.stats + row * 4);
    if constexpr (!AHEAD) load_pre(row);
    u32x4 yr[P];
    auto load_y = [&]() {
      const T *y = row_start<TEAM, T>(a.y, off), *g = row_start<TEAM, T>(a.gate, group * d);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N;
        yr[p] = zero;
        if (a.y) yr[p] = load_piece<T, R>(y, at, d);
        if constexpr (GATE != CHUNK)
          gr[p] = load_piece<T, R>(g, at, d);
      }
    };
    float D[P][N];
    {
      u32x4 dhr[P];
      auto load_rest = [&]() {
        const T* dh_out = row_start<TEAM, T>(a.dh_out, off);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          dhr[p] = zero;
          if (a.dh_out)
            dhr[p] = load_piece<T, R>(dh_out, (p * TEAM + lane) * N, d);
        }
        if constexpr (!LATE) load_y();
      };
      if constexpr (REREAD)
        load_pre_pars();
      else
        load_rest();
      float c1 = 0.0f, c2 = 0.0f;
      if (a.pre != MONARCH_NORM_NONE) {
        const float mean = st[2] * st[3];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float dn[N], h[N], w[N];
          PieceOf<T>::unpack(dnr[p], dn);
          if constexpr (R != WHOLE) mask<R, N>(dn, (p * TEAM + lane) * N, d);
          unpack_low<T>(hr[p], low_word(p), h);
          if constexpr (BIAS) s_preb.add(p, dn);
          forget(pre_wr[p]);
          PieceOf<T>::unpack(pre_wr[p], w);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            h[i] = fmaf(h[i], st[3], -mean) * dn[i];   // dn hhat
            s[0] = fmaf(h[i], w[i], s[0]);
            s[1] = fmaf(dn[i], w[i], s[1]);
          }
          s_pre.add(p, h);
        }
        if constexpr (REREAD) load_rest();
        team.template reduce<SumOp, 2>(s);
        // D = dh' + rho (q - hhat c1 - c2) with hhat = h rho - mean
        c1 = s[0] * inv_d;
        c2 = a.pre == MONARCH_NORM_LAYER ? s[1] * inv_d : 0.0f;
        const float k1 = c1 * st[3] * st[3], k0 = st[3] * (c2 - c1 * mean);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int at = (p * TEAM + lane) * N;
          float dn[N], h[N], w[N];
          forget(dnr[p]);
          forget(hr[p]);
          if constexpr (N == 8) forget(lowr[p]);
          forget(pre_wr[p]);
          PieceOf<T>::unpack(dnr[p], dn);
          unpack_low<T>(hr[p], low_word(p), h);
          PieceOf<T>::unpack(dhr[p], D[p]);
          PieceOf<T>::unpack(pre_wr[p], w);
#pragma unroll
          for (int i = 0; i < N; ++i)
            D[p][i] += fmaf(st[3] * dn[i], w[i], -fmaf(h[i], k1, k0));
          mask<R, N>(D[p], at, d);
        }
      } else {
        if constexpr (REREAD) load_rest();
#pragma unroll
        for (int p = 0; p < P; ++p) {
          PieceOf<T>::unpack(dhr[p], D[p]);
          if constexpr (R != WHOLE) mask<R, N>(D[p], (p * TEAM + lane) * N, d);
        }
      }
    }
    if constexpr (LATE) load_y();
    if constexpr (REREAD) load_post_pars();
    if (AHEAD && row + step < last) load_pre(row + step);
    T* dh = row_start<TEAM, T>(a.dh, off);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = (p * TEAM + lane) * N;
      if (at < d) {
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = a.skip * D[p][i];
        store_piece<T, R>(dh, at, d, PieceOf<T>::pack(o));
      }
    }
    if (a.y) {
      const float mean = st[0] * st[1];
      float s[2] = {0.0f, 0.0f};
      T *dgate = row_start<TEAM, T>(a.dgate, group * d), *dy = row_start<TEAM, T>(a.dy, off);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N;
        float y[N], w[N], g[N], o[N];
        PieceOf<T>::unpack(yr[p], y);
        forget(post_wr[p]);
        forget(gr[p]);
        PieceOf<T>::unpack(post_wr[p], w);
        PieceOf<T>::unpack(gr[p], g);
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = fmaf(y[i], st[1], -mean);   // yhat
        if constexpr (GATE != CHUNK) {
          // dgate = branch D u
          float b[N];
          if constexpr (BIAS)
            PieceOf<T>::unpack(par_piece<T, R>(a.post_b, 0, at, d, 0.0f), b);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = D[p][i] * (BIAS ? fmaf(y[i], w[i], b[i]) : y[i] * w[i]);
          if constexpr (GATE == RUN) {
            s_gate.add(p, o);
          } else if (a.dgate) {
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] *= a.branch;
            store_piece<T, R>(dgate, at, d, PieceOf<T>::pack(o));
          }
          // e / branch = g D, which D becomes
#pragma unroll
          for (int i = 0; i < N; ++i) D[p][i] *= g[i];
        }
        if constexpr (BIAS) s_postb.add(p, D[p]);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = D[p][i] * y[i];
        s_post.add(p, o);
        // D becomes q2 = branch g D w
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if constexpr (GATE == CHUNK) D[p][i] *= g[i];
          D[p][i] *= a.branch * w[i];
          s[0] = fmaf(D[p][i], y[i], s[0]);
          s[1] += D[p][i];
        }
      }
      float k1 = 0.0f, k0 = 0.0f;
      if (a.post != MONARCH_NORM_NONE) {
        team.template reduce<SumOp, 2>(s);
        // dy = rho (q2 - yhat c1 - c2) with yhat = y rho - mean
        const float c1 = s[0] * inv_d, c2 = a.post == MONARCH_NORM_LAYER ? s[1] * inv_d : 0.0f;
        k1 = c1 * st[1] * st[1];
        k0 = st[1] * (c2 - c1 * mean);
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N;
        float y[N];
        forget(yr[p]);
        PieceOf<T>::unpack(yr[p], y);
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = fmaf(st[1], D[p][i], -fmaf(y[i], k1, k0));
        store_piece<T, R>(dy, at, d, PieceOf<T>::pack(y));
      }
    }
    if constexpr (GATE == TOKEN) ++group;
    if constexpr (GATE == RUN) {
      if (--left == 0) {
        left = a.rows_per_gate;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int at = (p * TEAM + lane) * N;
          float o[N];
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = a.branch * s_gate.v[p][i];
          if (a.dgate)
            store_piece<T, R>(static_cast<T*>(a.dgate) + group * d, at, d, PieceOf<T>::pack(o));
        }
        s_gate.clear(nullptr);
        ++group;
      }
    }
  }
  // this chunk's sums: the teams' are added in team order. `shift` is how far a
  // piece is moved back to end with its row (load_piece).
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.sums * a.d;
  auto shift = [&](int at) { return R == WHOLE ? 0 : max(at + N - a.d, 0); };
  auto put = [&](int which, const auto& s) {
    if (which < 0) return;
    float* out = part + static_cast<int64_t>(which) * a.d;
    if constexpr (std::is_same<decltype(s), const Sums<WG, P, N, true>&>::value) {
      __syncthreads();
      for (int at = threadIdx.x; at < a.d; at += WG) {
        const int p = at / (TEAM * N), l = at / N % TEAM, i = at % N + shift(at / N * N);
        float t = s.at(p, i, l);
#pragma unroll
        for (int k = 1; k < TEAMS; ++k) t += s.at(p, i, k * TEAM + l);
        out[at] = t;
      }
    } else {
      float* to = TEAMS == 1 ? out : reinterpret_cast<float*>(shared) + tm * COLS;
      if constexpr (TEAMS > 1) __syncthreads();
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * TEAM + lane) * N, back = shift(at);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (at < a.d && i >= back) to[at - back + i] = s.v[p][i];
      }
      if constexpr (TEAMS > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += WG) {
          const float* from = reinterpret_cast<const float*>(shared) + c;
          float t = from[0];
#pragma unroll
          for (int k = 1; k < TEAMS; ++k) t += from[k * COLS];
          out[c] = t;
        }
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

// Joins the chunks' sums (SandwichJoin).
constexpr int JC = 32, JS = 32;

template <typename T>
__global__ __launch_bounds__(JC* JS) void sandwich_join_kernel(SandwichJoin a) {
  __shared__ float buf[2][JS][JC];
  const int col = threadIdx.x % JC, slice = threadIdx.x / JC;
  const int at = blockIdx.y * JC + col;
  const int64_t job = blockIdx.x;
  int which, which2 = -1;
  int c0 = 0, c1 = a.chunks;
  bool gated = false;
  void* out;
  if (job < kWeightJobs) {
    which = job == 0 ? a.s_post : job == 1 ? a.s_postb : job == 2 ? a.s_pre : a.s_preb;
    out = job == 0 ? a.dpost_w : job == 1 ? a.dpost_b : job == 2 ? a.dpre_w : a.dpre_b;
    gated = job < 2 && a.gate;
  } else {
    which = a.s_post;
    which2 = a.post_b ? a.s_postb : -1;
    c0 = static_cast<int>(job - kWeightJobs) * a.cpg;
    c1 = c0 + a.cpg;
    out = static_cast<T*>(a.dgate) + (job - kWeightJobs) * a.d;
  }
  if (!out || which < 0) return;   // the whole workgroup
  const int per = (c1 - c0 + JS - 1) / JS;
  const int b = c0 + slice * per, e = min(b + per, c1);
  float s = 0.0f, s2 = 0.0f;
  if (at < a.d) {
    const int64_t stride = static_cast<int64_t>(a.sums) * a.d;
    const float* p = a.part + static_cast<int64_t>(which) * a.d + at;
    const float* p2 = a.part + static_cast<int64_t>(which2 < 0 ? which : which2) * a.d + at;
    if (which2 >= 0) {
#pragma unroll 8
      for (int c = b; c < e; ++c) {
        s += p[c * stride];
        s2 += p2[c * stride];
      }
    } else if (!gated) {
#pragma unroll 8
      for (int c = b; c < e; ++c) s += p[c * stride];
    } else {
      int c = b;
      while (c < e) {   // the chunks of one gate row at a time
        const int g = c / a.cpg, end = min(e, (g + 1) * a.cpg);
        float t = 0.0f;
#pragma unroll 8
        for (; c < end; ++c) t += p[c * stride];
        s = fmaf(t, Io<T>::load(a.gate, static_cast<int64_t>(g) * a.d + at), s);
      }
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
  Io<T>::store(out, at, s);
}

// ----------------------------------------------------------------- launches

// How rows of d elements lie.
template <typename T> Rows rows_of(int64_t d) {
  constexpr int n = PieceOf<T>::N;
  return d % n == 0 ? WHOLE : d > n ? CUT : SHORT;
}

template <typename T, int TEAM, int P>
void fwd_launch(const SandwichFwd& a, Rows lie, hipStream_t s) {
  constexpr int WG = TEAM > 64 ? TEAM : 256, TEAMS = WG / TEAM;
  // one row a team, or the workgroups that fit the chip at once where they load
  // ahead; 2^20 workgroups are fewer than 2^32 threads
  const int64_t most = TEAM == 1024 ? kSandwichCus : 1 << 20;
  int64_t grid = (a.rows + TEAMS - 1) / TEAMS;
  if (grid > most) grid = most;
  const dim3 g(static_cast<unsigned>(grid)), block(WG);
  // odd widths: without biases' code nothing was gained (4096 x 4095 bf16 28.9 us
  // against 29.7, 65536 x 250 32.6 against 30.9)
  if (lie == CUT) {
    hipLaunchKernelGGL((sandwich_fwd_kernel<T, TEAM, P, true, CUT>), g, block, 0, s, a);
  } else if (lie == SHORT) {
    if constexpr (TEAM == 16 && P == 1)
      hipLaunchKernelGGL((sandwich_fwd_kernel<T, TEAM, P, true, SHORT>), g, block, 0, s, a);
  } else if (a.post_b || a.pre_b) {
    hipLaunchKernelGGL((sandwich_fwd_kernel<T, TEAM, P, true, WHOLE>), g, block, 0, s, a);
  } else {
    hipLaunchKernelGGL((sandwich_fwd_kernel<T, TEAM, P, false, WHOLE>), g, block, 0, s, a);
  }
}

template <typename T, int TEAM, int P>
void bwd_launch(const SandwichBwd& a, const SandwichBwdPlan& p, Rows lie, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.chunks)), block(TEAM > 64 ? TEAM : 256);
#define BWD_GO(GATE, BIAS, ROWS) \
  hipLaunchKernelGGL((sandwich_bwd_kernel<T, TEAM, P, GATE, BIAS, ROWS>), grid, block, 0, s, a)
#define BWD_ANY(ROWS)                                        \
  switch (p.gate * 2 + (p.bias ? 1 : 0)) {                   \
    case CHUNK * 2: BWD_GO(CHUNK, false, ROWS); break;       \
    case CHUNK * 2 + 1: BWD_GO(CHUNK, true, ROWS); break;    \
    case RUN * 2: BWD_GO(RUN, false, ROWS); break;           \
    case RUN * 2 + 1: BWD_GO(RUN, true, ROWS); break;        \
    case TOKEN * 2: BWD_GO(TOKEN, false, ROWS); break;       \
    default: BWD_GO(TOKEN, true, ROWS); break;               \
  }
  // Odd widths have all six kernels too, against one for biases and any gate run. A
  // gate a row, before and after: 16384 x 767 bf16 66 and 52 us (with biases 71 and 58),
  // 2048 x 16383 bf16 385 and 145, 2048 x 12001 fp32 191 and 172. It costs rows of about 1000
  // features with biases a little: 16384 x 1023 bf16 73 and 77, 625 fp32 46.4 and 48.2.
  if (lie == WHOLE) {
    BWD_ANY(WHOLE)
  } else if (lie == CUT) {
    BWD_ANY(CUT)
  } else if constexpr (TEAM == 32 && P == 1) {
    // rows of a few bytes: one kernel for any gate run and any bias
    if (p.gate == CHUNK)
      BWD_GO(CHUNK, true, SHORT);
    else
      BWD_GO(RUN, true, SHORT);
  }
#undef BWD_ANY
#undef BWD_GO
}

}  // namespace

#define TEAM_CASE(CALL, T, TEAM, P)                \
  case (TEAM) * 8 + (P): CALL(T, TEAM, P); break;

// The pairs (team, pieces) that the two shape functions give.
template <typename T> hipError_t sandwich_launch_fwd(const SandwichFwd& a, hipStream_t s) {
  const Shape sh = sandwich_fwd_shape(a.d, sizeof(T) == 2);
  const Rows lie = rows_of<T>(a.d);
#define FWD(T, TEAM, P) fwd_launch<T, TEAM, P>(a, lie, s)
  if constexpr (sizeof(T) == 2) {
    switch (sh.team * 8 + sh.pieces) {
      TEAM_CASE(FWD, T, 16, 1)
      TEAM_CASE(FWD, T, 16, 2)
      TEAM_CASE(FWD, T, 16, 3)
      TEAM_CASE(FWD, T, 32, 2)
      TEAM_CASE(FWD, T, 32, 3)
      TEAM_CASE(FWD, T, 64, 2)
      TEAM_CASE(FWD, T, 64, 3)
      TEAM_CASE(FWD, T, 128, 2)
      TEAM_CASE(FWD, T, 256, 2)
      TEAM_CASE(FWD, T, 512, 2)
      TEAM_CASE(FWD, T, 1024, 2)
      default: return hipErrorInvalidConfiguration;
    }
  } else {
    switch (sh.team * 8 + sh.pieces) {
      TEAM_CASE(FWD, T, 16, 1)
      TEAM_CASE(FWD, T, 16, 2)
      TEAM_CASE(FWD, T, 16, 3)
      TEAM_CASE(FWD, T, 16, 4)
      TEAM_CASE(FWD, T, 32, 3)
      TEAM_CASE(FWD, T, 32, 4)
      TEAM_CASE(FWD, T, 64, 3)
      TEAM_CASE(FWD, T, 64, 4)
      TEAM_CASE(FWD, T, 128, 3)
      TEAM_CASE(FWD, T, 128, 4)
      TEAM_CASE(FWD, T, 256, 3)
      TEAM_CASE(FWD, T, 256, 4)
      TEAM_CASE(FWD, T, 512, 3)
      TEAM_CASE(FWD, T, 512, 4)
      TEAM_CASE(FWD, T, 1024, 3)
      TEAM_CASE(FWD, T, 1024, 4)
      default: return hipErrorInvalidConfiguration;
    }
  }
#undef FWD
  return hipGetLastError();
}

template <typename T>
hipError_t sandwich_launch_bwd(const SandwichBwd& a, const SandwichBwdPlan& p, hipStream_t s) {
  const Rows lie = rows_of<T>(a.d);
#define BWD(T, TEAM, P) bwd_launch<T, TEAM, P>(a, p, lie, s)
  if constexpr (sizeof(T) == 2) {
    switch (p.shape.team * 8 + p.shape.pieces) {
      TEAM_CASE(BWD, T, 32, 1)
      TEAM_CASE(BWD, T, 32, 2)
      TEAM_CASE(BWD, T, 32, 3)
      TEAM_CASE(BWD, T, 64, 2)
      TEAM_CASE(BWD, T, 64, 3)
      TEAM_CASE(BWD, T, 128, 2)
      TEAM_CASE(BWD, T, 256, 2)
      TEAM_CASE(BWD, T, 512, 2)
      TEAM_CASE(BWD, T, 512, 3)
      TEAM_CASE(BWD, T, 512, 4)
      default: return hipErrorInvalidConfiguration;
    }
  } else {
    switch (p.shape.team * 8 + p.shape.pieces) {
      TEAM_CASE(BWD, T, 32, 1)
      TEAM_CASE(BWD, T, 32, 2)
      TEAM_CASE(BWD, T, 32, 3)
      TEAM_CASE(BWD, T, 32, 4)
      TEAM_CASE(BWD, T, 64, 3)
      TEAM_CASE(BWD, T, 64, 4)
      TEAM_CASE(BWD, T, 128, 3)
      TEAM_CASE(BWD, T, 128, 4)
      TEAM_CASE(BWD, T, 256, 3)
      TEAM_CASE(BWD, T, 256, 4)
      TEAM_CASE(BWD, T, 512, 3)
      TEAM_CASE(BWD, T, 512, 4)
      TEAM_CASE(BWD, T, 1024, 3)
      TEAM_CASE(BWD, T, 1024, 4)
      default: return hipErrorInvalidConfiguration;
    }
  }
#undef BWD
  return hipGetLastError();
}
#undef TEAM_CASE

template <typename T>
hipError_t sandwich_launch_join(const SandwichJoin& a, int64_t jobs, hipStream_t s) {
  // gate rows that are joined here are fewer than the teams of a launch (bwd_plan)
  const dim3 grid(static_cast<unsigned>(jobs), static_cast<unsigned>((a.d + JC - 1) / JC));
  hipLaunchKernelGGL((sandwich_join_kernel<T>), grid, dim3(JC * JS), 0, s, a);
  return hipGetLastError();
}

}  // namespace monarch
