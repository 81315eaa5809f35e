// Head loss: the loss of rows x [n][d] under a dense head w [vocab][d] and its
// gradients by both, in pieces of the vocabulary; the logits z = x w^T are not kept (but those of
// up to 32 rows for the length of a step).
//
// With q = softmax(z / T), s = softmax(z), p = softmax(t / T) over a row's valid teacher
// entries (id_k, t_k), label c and row weight r:
//   loss = mix T^2 sum_k p_k (log p_k - log q[id_k]) - (1 - mix) log s[c]
//   g_v  = r (mix T (q_v - sum_{k: id_k = v} p_k) + (1 - mix) (s_v - [v = c]))
//   dx = g w, dw = g^T x
//
// A forward pass takes every tile of logits from its product to (maximum, sum at T,
// sum at 1) of its rows, and joins these over the tiles. A backward pass knows the sums,
// so it computes the logits again, a piece of the vocabulary at a time, turns them into
// g in the product's epilogue, writes that piece of g to the workspace and multiplies
// it twice. Rows that count nothing (no label, no entry) are left out of all products:
// the rows that do are first copied side by side, with their columns padded to whole K
// tiles; what a row left out holds (NaN too) reaches nothing.
//
// In bf16 g is divided by the largest weight of a row and multiplied back in its products' fp32 sums: the
// labels' elements, nearly all of g, are then 1 - s[c] or a little less, whose rounding to bf16 is
// half of that of a value just over a power of two (as 1 / rows may be, alike for every row). Up to 64 rows, where
// single roundings do not average out, g is held in two bf16 parts: the second one's rows lie behind the first's
// (32 or 64 of them), x's rows are copied twice, and the products take them as that many more rows: dw's K tiles and dx's
// output tiles have the room, and the head is read no more often.
//
// The teacher's columns of g are few: their logits are taken from products of their
// own in the forward pass (a wave an entry), and each is written again behind the piece's
// epilogue with its share of p, once, in fp32 up to its one rounding.
#include <math.h>
#include <stdio.h>

#include "api_internal.h"
#include "head.h"
#include "kernels.h"
#include "monarch.h"
#include "team.h"

namespace monarch {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int64_t kMaxFeatures = int64_t(1) << 20;
// Of g. Steps with pieces of at most 2 GiB, 1 GiB, 512 and 256 MiB, ms: 16384 x 768 x 50257 bf16 5.36, 5.26, 5.56, 5.66;
// 4096 x 4096 x 131072 14.75, 14.66, 14.91, 15.31; 65536 x 1024 x 131072 68.5, 68.0, 71.1, 75.9; 4096 x 768 x 50257 fp32
// 5.54, 5.63, 5.75, 5.89.
constexpr int64_t kPieceBytes = int64_t(1) << 30;

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The rows in use.
struct Rows {
  int* count;
  int* idx;      // [np] row of x
  int* pos;      // [rows] place among them, -1
  int* label;    // [np] label, -1 without one
  int* has;      // [np] whether the row has a valid entry
  int* flag;     // [rows] whether it has (before the rows are counted)
  float* scale;  // what g is divided by
  int* g_rows;   // rows of g in use
  int fold;      // 0, or the rows of one of g's two parts
};

struct Call {
  const void* x;
  const void* w;
  const float* teacher;
  const int64_t* ids;
  const int64_t* labels;
  const float* weight;        // null: 1
  float *loss, *stats;
  void *dx, *dw;
  int64_t rows, ldx, d, vocab;
  int top;
  float temperature, mix;     // temperature 1 where there is no first term
  bool bf16, told, taught;
  HeadSecond second;
};

__device__ __forceinline__ bool entry_ok(int64_t id, float t, int64_t vocab) {
  return id >= 0 && id < vocab && t > -INFINITY;
}

// A row of d bf16 elements copied to dp, zeros behind them (or zeros throughout), by N threads.
template <int N>
__device__ __forceinline__ void copy_row(const uint16_t* s, bool zero, int64_t d, int64_t dp, uint16_t* o, int t) {
  const bool whole = ((reinterpret_cast<uintptr_t>(s) & 15) == 0) && d % 8 == 0;
  for (int64_t e = t * 8; e < dp; e += N * 8) {
    u32x4 v = {0, 0, 0, 0};
    if (!zero && e < d) {
      if (whole) {
        v = *reinterpret_cast<const u32x4*>(s + e);
      } else {
        uint16_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = e + i < d ? s[e + i] : uint16_t(0);
        __builtin_memcpy(&v, h, 16);
      }
    }
    *reinterpret_cast<u32x4*>(o + e) = v;
  }
}

// A wave a row: does it have an entry? (`group`, here and below: this launch's first workgroup.)
__global__ __launch_bounds__(256) void head_flag_kernel(Call c, Rows r, int64_t group) {
  const int64_t i = (group + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (i >= c.rows) return;
  bool any = false;
  for (int k = threadIdx.x & 63; k < c.top; k += 64)
    any |= entry_ok(c.ids[i * c.top + k], c.teacher[i * c.top + k], c.vocab);
  const bool all = __any(any);
  if ((threadIdx.x & 63) == 0) r.flag[i] = all;
}

// One workgroup: the rows in use, in their order; loss and statistics of the others are 0.
// With xc (few rows in bf16) it copies them too, as head_copy_kernel would.
__global__ __launch_bounds__(1024) void head_rows_kernel(Call c, Rows r, uint32_t* zeros, uint16_t* xc, int64_t dp) {
  constexpr int PER = 4;
  __shared__ int s_wave[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (threadIdx.x < 4) zeros[threadIdx.x] = 0;
  int base = 0;
  float most = 0.f;   // weight of a row in use
  for (int64_t first = 0; first < c.rows; first += 1024 * PER) {
    int label[PER], has[PER], mine = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int64_t i = first + threadIdx.x * PER + e;
      label[e] = -1, has[e] = 0;
      if (i < c.rows) {
        if (c.told) {
          const int64_t l = c.labels[i];
          if (l >= 0 && l < c.vocab) label[e] = static_cast<int>(l);
        }
        if (c.taught) has[e] = r.flag[i];
      }
      mine += label[e] >= 0 || has[e];
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    if (lane == 63) s_wave[wave] = upto;
    __syncthreads();
    int at = base + upto - mine, all = base;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      if (w < wave) at += s_wave[w];
      all += s_wave[w];
    }
    base = all;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int64_t i = first + threadIdx.x * PER + e;
      if (i >= c.rows) continue;
      const bool used = label[e] >= 0 || has[e];
      r.pos[i] = used ? at : -1;
      if (used) {
        const float w = c.weight ? fabsf(c.weight[i]) : 1.f;
        if (isfinite(w)) most = fmaxf(most, w);
        r.idx[at] = static_cast<int>(i), r.label[at] = label[e], r.has[at] = has[e];
        ++at;
      } else if (c.loss) {
        c.loss[i] = 0.f;
        *reinterpret_cast<f32x4*>(c.stats + i * 4) = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    __syncthreads();
  }
  // the last tile's other rows
  const int end = (base + static_cast<int>(kHeadRows) - 1) / static_cast<int>(kHeadRows) * static_cast<int>(kHeadRows);
  for (int k = base + threadIdx.x; k < end; k += 1024) r.idx[k] = 0, r.label[k] = -1, r.has[k] = 0;
  most = lanes_reduce<MaxOp, 64>(most);
  __shared__ float s_most[16];
  if (lane == 0) s_most[wave] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    *r.count = base;
    *r.g_rows = r.fold && base > 0 ? 2 * r.fold : base;
    for (int w = 0; w < 16; ++w) most = fmaxf(most, s_most[w]);
    most *= fmaxf(c.told ? 1.0f - c.mix : 0.f, c.taught ? c.mix * c.temperature : 0.f);
    *r.scale = c.bf16 && most > 1e-30f && most < 1e30f ? most : 1.f;
  }
  if (xc) {
    __syncthreads();
    // a wave a row at a time, both parts' rows of g
    for (int k = wave; k < 2 * r.fold; k += 16) {
      const int from = k % r.fold;
      copy_row<64>(static_cast<const uint16_t*>(c.x) + (from < base ? r.idx[from] : 0) * c.ldx, from >= base, c.d, dp, xc + k * dp, lane);
    }
  }
}

// One value as bf16, and what is left of it.
__device__ __forceinline__ uint16_t next_part(float& v) {
  const uint16_t h = f32_to_bf16(finite_bf16(v));
  v = isfinite(v) ? v - bf16_to_f32(h) : 0.f;
  return h;
}

// Rows of d elements copied to rows of dp, zeros behind them; fp32 as three bf16 planes.
// With idx the rows are idx[k] for k < *count, then zeros up to the next whole tile (with
// fold, the first `fold` of these twice); without, k for k < rows, zeros behind. A workgroup a row.
template <typename T>
__global__ __launch_bounds__(256) void head_copy_kernel(const T* __restrict__ src, int64_t ld, const int* idx,
                                                        const int* count, int fold, int64_t rows, int64_t d, int64_t dp,
                                                        uint16_t* __restrict__ dst, int64_t plane, int64_t group) {
  constexpr bool F32 = sizeof(T) == 4;
  const int64_t to = group + blockIdx.x, k = fold && to < 2 * fold ? to % fold : to;
  bool zero = k >= rows;
  int64_t row = zero ? 0 : k;
  if (idx) {
    const int n = *count;
    if (to >= (n + kHeadRows - 1) / kHeadRows * kHeadRows) return;
    zero = k >= n;
    row = zero ? 0 : idx[k];
  }
  const T* s = src + row * ld;
  uint16_t* o = dst + to * dp;
  if constexpr (F32) {
    const bool whole = ((reinterpret_cast<uintptr_t>(s) & 15) == 0) && d % 4 == 0;
    for (int64_t e = threadIdx.x * 4; e < dp; e += 1024) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (!zero && e < d) {
        if (whole) {
          const f32x4 q = *reinterpret_cast<const f32x4*>(s + e);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = q[i];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < d) v[i] = s[e + i];
        }
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = next_part(v[i]);
        __builtin_memcpy(o + p * plane + e, h, 8);
      }
    }
  } else {
    copy_row<256>(s, zero, d, dp, o, threadIdx.x);
  }
}

// Logits of the teacher's entries: a wave takes four of a row at a time. Stored by row
// of x behind the statistics; 0 for an entry that is not valid.
template <typename T>
__global__ __launch_bounds__(256) void head_entries_kernel(Call c, Rows r, const T* __restrict__ xs, int64_t ldx,
                                                           bool by_row, const T* __restrict__ ws, int64_t ldw,
                                                           int64_t group) {
  const int64_t k = group + blockIdx.x;
  if (k >= *r.count || !r.has[k]) return;
  const int64_t i = r.idx[k];
  const T* x = xs + (by_row ? i : k) * ldx;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* out = c.stats + c.rows * 4 + i * c.top;
  for (int j0 = wave * 4; j0 < c.top; j0 += 16) {
    const T* w[4];
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    bool ok[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + e < c.top ? j0 + e : c.top - 1;
      const int64_t id = c.ids[i * c.top + j];
      ok[e] = entry_ok(id, c.teacher[i * c.top + j], c.vocab);
      w[e] = ws + (ok[e] ? id : 0) * ldw;
    }
    if constexpr (sizeof(T) == 2) {
      for (int64_t at = lane * 8; at < c.d; at += 512) {
        // rows of the head in place are whole pieces; padded copies end in zeros
        float a[8];
        PieceOf<uint16_t>::unpack(*reinterpret_cast<const u32x4*>(x + at), a);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float b[8];
          PieceOf<uint16_t>::unpack(*reinterpret_cast<const u32x4*>(w[e] + at), b);
#pragma unroll
          for (int q = 0; q < 8; ++q) sum[e] = fmaf(a[q], b[q], sum[e]);
        }
      }
    } else {
      if (c.d % 4 == 0) {   // the head's rows start at 16 bytes, x's at any element
        for (int64_t at = lane * 4; at < c.d; at += 256) {
          const float a[4] = {x[at], x[at + 1], x[at + 2], x[at + 3]};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f32x4 b = *reinterpret_cast<const f32x4*>(w[e] + at);
#pragma unroll
            for (int q = 0; q < 4; ++q) sum[e] = fmaf(a[q], b[q], sum[e]);
          }
        }
      } else {
        for (int64_t at = lane; at < c.d; at += 64) {
          const float a = x[at];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = fmaf(a, w[e][at], sum[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s = lanes_reduce<SumOp, 64>(sum[e]);
      if (lane == 0 && j0 + e < c.top) out[j0 + e] = ok[e] ? s : 0.f;
    }
  }
}

// Maximum and logarithm of the sum of exp(t / T) over a row's valid entries, by one wave.
__device__ __forceinline__ void teacher_sums(const Call& c, int64_t i, int lane, float* top, float* sum) {
  const float ct = kLog2e / c.temperature;
  float m = -3.402823466e38f;
  for (int j = lane; j < c.top; j += 64)
    if (entry_ok(c.ids[i * c.top + j], c.teacher[i * c.top + j], c.vocab)) m = fmaxf(m, c.teacher[i * c.top + j]);
  m = lanes_reduce<MaxOp, 64>(m);
  float s = 0.f;
  for (int j = lane; j < c.top; j += 64)
    if (entry_ok(c.ids[i * c.top + j], c.teacher[i * c.top + j], c.vocab)) s += exp2_of((c.teacher[i * c.top + j] - m) * ct);
  *top = m;
  *sum = lanes_reduce<SumOp, 64>(s);
}

// The factors for g of row k (compact), from its largest logit and sums.
__device__ __forceinline__ void row_factors(const Call& c, const Rows& r, int64_t k, int64_t i, float m, float st, float s1,
                                            HeadRow* out, float* taught) {
  HeadRow o;
  const float w = (c.weight ? c.weight[i] : 1.0f) / *r.scale;
  const float a = r.has[k] ? c.mix * c.temperature * w : 0.f;
  o.m = m;
  o.off = r.label[k] >= 0 ? (1.0f - c.mix) * w : 0.f;
  // one softmax at T = 1, or with one of the two terms alone
  const bool one = c.second == HEAD_ONE;
  o.a = one ? (a + o.off) / st : a / st;
  o.b = one ? 0.f : o.off / s1;
  out[k] = o;
  taught[k] = a;
}

// Joins the tiles' sums of RW rows a workgroup, and gives the rows' losses; in a step their factors for g
// too, as head_factors_kernel.
template <int RW>
__global__ __launch_bounds__(256) void head_loss_kernel(Call c, Rows r, const float* __restrict__ part, int64_t np,
                                                        int tiles, const float* __restrict__ z_label, HeadRow* factors,
                                                        float* taught, int64_t group) {
  constexpr int SL = 256 / RW;
  __shared__ float s[3][256];
  const int64_t k0 = (group + blockIdx.x) * RW;
  const int count = *r.count;
  if (k0 >= count) {
    if (factors && k0 < (count + kHeadRows - 1) / kHeadRows * kHeadRows && threadIdx.x < RW)
      factors[k0 + threadIdx.x] = HeadRow{0.f, 0.f, 0.f, 0.f}, taught[k0 + threadIdx.x] = 0.f;
    return;
  }
  const float ct = kLog2e / c.temperature;
  const int col = threadIdx.x % RW, slice = threadIdx.x / RW;
  const float* at = part + k0 + col;
  float m = -3.402823466e38f, st = 0.f, s1 = 0.f;
  // in fixed order: tiles slice, slice + SL, ...
  for (int t = slice; t < tiles; t += SL) {
    const float* o = at + static_cast<int64_t>(t) * 3 * np;
    const float tm = o[0], ts = o[np], t1 = o[2 * np];
    const float to = fmaxf(m, tm), f = m - to, g = tm - to;
    st = st * exp2_of(f * ct) + ts * exp2_of(g * ct);
    s1 = s1 * exp2_of(f * kLog2e) + t1 * exp2_of(g * kLog2e);
    m = to;
  }
  s[0][threadIdx.x] = m, s[1][threadIdx.x] = st, s[2][threadIdx.x] = s1;
  for (int half = SL / 2; half > 0; half /= 2) {
    __syncthreads();
    if (slice < half) {
      const int u = threadIdx.x + half * RW;
      const float tm = s[0][u], to = fmaxf(m, tm), f = m - to, g = tm - to;
      st = st * exp2_of(f * ct) + s[1][u] * exp2_of(g * ct);
      s1 = s1 * exp2_of(f * kLog2e) + s[2][u] * exp2_of(g * kLog2e);
      m = to;
      s[0][threadIdx.x] = m, s[1][threadIdx.x] = st, s[2][threadIdx.x] = s1;
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 63;
  for (int w = threadIdx.x >> 6; w < RW; w += 4) {
    const int64_t k = k0 + w;
    if (k >= count) {
      if (factors && lane == 0) factors[k] = HeadRow{0.f, 0.f, 0.f, 0.f}, taught[k] = 0.f;
      continue;
    }
    const int64_t i = r.idx[k];
    const float rm = s[0][w], rt = s[1][w], r1 = s[2][w];
    float loss = 0.f;
    if (r.has[k]) {
      float tm, ts;
      teacher_sums(c, i, lane, &tm, &ts);
      const float log_ts = logf(ts), log_q = logf(rt), by = 1.0f / c.temperature;
      float kl = 0.f;
      for (int j = lane; j < c.top; j += 64) {
        const float t = c.teacher[i * c.top + j];
        if (!entry_ok(c.ids[i * c.top + j], t, c.vocab)) continue;
        const float e = exp2_of((t - tm) * (kLog2e * by)), p = e / ts;
        const float z = c.stats[c.rows * 4 + i * c.top + j];
        if (p > 0.f) kl += p * (((t - tm) * by - log_ts) - ((z - rm) * by - log_q));
      }
      loss = c.mix * c.temperature * c.temperature * lanes_reduce<SumOp, 64>(kl);
    }
    if (r.label[k] >= 0) loss += (1.0f - c.mix) * (logf(r1) - (z_label[k] - rm));
    if (lane == 0) {
      c.loss[i] = loss;
      *reinterpret_cast<f32x4*>(c.stats + i * 4) = f32x4{rm, rt, r1, 0.f};
      if (factors) row_factors(c, r, k, i, rm, rt, r1, factors, taught);
    }
  }
}

// The rows' factors for g, from the forward pass's statistics (0 for the last tile's other rows).
__global__ __launch_bounds__(256) void head_factors_kernel(Call c, Rows r, HeadRow* out, float* taught) {
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int count = *r.count;
  if (k >= (count + kHeadRows - 1) / kHeadRows * kHeadRows) return;
  if (k < count) {
    const int64_t i = r.idx[k];
    const f32x4 st = *reinterpret_cast<const f32x4*>(c.stats + i * 4);
    row_factors(c, r, k, i, st[0], st[1], st[2], out, taught);
  } else {
    out[k] = HeadRow{0.f, 0.f, 0.f, 0.f};
    taught[k] = 0.f;
  }
}

// g of few rows (HEAD_THIN) from their logits, which a step keeps for its length: they are smaller than
// the head, which would be read again for them. Four words a thread, kThinRows rows.
__global__ __launch_bounds__(256) void head_few_kernel(Call c, Rows r, const HeadRow* __restrict__ rows,
                                                       const float* __restrict__ z, uint16_t* __restrict__ g, float* __restrict__ gf,
                                                       int64_t vp, int64_t plane) {
  const int64_t v = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  const int n = blockIdx.y;
  if (v >= vp) return;
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  if (n < *r.count) {
    const HeadRow h = rows[n];
    const f32x4 l = *reinterpret_cast<const f32x4*>(z + n * vp + v);
    const float ct = kLog2e / c.temperature;
    const int64_t own = r.label[n] - v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = c.second == HEAD_ONE   ? head_g<HEAD_ONE>(h, l[i], ct, own == i)
             : c.second == HEAD_OWN ? head_g<HEAD_OWN>(h, l[i], ct, own == i)
                                    : head_g<HEAD_SQUARE>(h, l[i], ct, own == i);
      if (v + i >= c.vocab) o[i] = 0.f;
    }
  }
  if (gf) {
    *reinterpret_cast<f32x4*>(gf + n * vp + v) = f32x4{o[0], o[1], o[2], o[3]};
    return;
  }
  uint16_t* to = g + n * vp + v;
  for (int q = 0; q < 2; ++q, to += plane) {
    uint16_t part[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i] = next_part(o[i]);
    __builtin_memcpy(to, part, 8);
  }
}

// The teacher's columns of a piece of g: a wave a row.
__global__ __launch_bounds__(64) void head_taught_kernel(Call c, Rows r, const HeadRow* __restrict__ rows,
                                                         const float* __restrict__ taught, uint16_t* __restrict__ g,
                                                         float* __restrict__ gf, int64_t vp, int64_t plane, int planes, int64_t v0, int64_t v1,
                                                         int64_t group) {
  extern __shared__ __align__(16) int s_id[];
  float* s_p = reinterpret_cast<float*>(s_id + c.top);
  const int64_t k = group + blockIdx.x;
  if (k >= *r.count || !r.has[k]) return;
  const int64_t i = r.idx[k];
  const int lane = threadIdx.x;
  float tm, ts;
  teacher_sums(c, i, lane, &tm, &ts);
  const float ct = kLog2e / c.temperature;
  for (int j = lane; j < c.top; j += 64) {
    const int64_t id = c.ids[i * c.top + j];
    const float t = c.teacher[i * c.top + j];
    const bool ok = entry_ok(id, t, c.vocab);
    s_id[j] = ok ? static_cast<int>(id) : -1;
    s_p[j] = ok ? exp2_of((t - tm) * ct) / ts : 0.f;
  }
  __syncthreads();
  const HeadRow h = rows[k];
  const int label = r.label[k];
  for (int j = lane; j < c.top; j += 64) {
    const int id = s_id[j];
    if (id < v0 || id >= v1) continue;
    // entries that name one word: the first writes their sum
    float p = 0.f;
    bool first = true;
    for (int u = 0; u < c.top; ++u)
      if (s_id[u] == id) {
        first &= u >= j;
        p += s_p[u];
      }
    if (!first) continue;
    const float z = c.stats[c.rows * 4 + i * c.top + j] - h.m;
    float v = h.a * exp2_of(z * ct) + (c.second != HEAD_ONE ? h.b * exp2_of(z * kLog2e) : 0.f) - taught[k] * p;
    if (id == label) v -= h.off;
    if (gf) {
      gf[k * vp + (id - v0)] = v;
      continue;
    }
    uint16_t* o = g + k * vp + (id - v0);
    for (int q = 0; q < planes; ++q) o[q * plane] = next_part(v);
  }
}

// dx of every row from the splits' sums; rows left out get 0. Four columns a thread, SL threads
// that share the splits (many of them, where rows are few: 64 splits of 8 x 768 11 us with one thread, 5 with 16).
template <typename T, int SL>
__global__ __launch_bounds__(256) void head_dx_out_kernel(const float* __restrict__ part, const int* __restrict__ pos,
                                                          int64_t rows, int64_t np, int64_t d, int64_t dp, int splits,   // part [splits][np][dp]
                                                          int fold, const float* __restrict__ scale, T* __restrict__ dx,
                                                          int64_t group) {
  constexpr int OUT = 256 / SL;
  const int64_t per = (d + 3) / 4, at = (group + blockIdx.x) * OUT + threadIdx.x % OUT;
  const int slice = threadIdx.x / OUT;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  int64_t i = 0, e = 0;
  const bool in = at < rows * per;
  if (in) {
    i = at / per, e = (at - i * per) * 4;
    const int64_t k = pos[i];
    if (k >= 0)
      for (int s = slice; s < splits; s += SL) {
        v += *reinterpret_cast<const f32x4*>(part + (s * np + k) * dp + e);
        if (fold) v += *reinterpret_cast<const f32x4*>(part + (s * np + k + fold) * dp + e);
      }
  }
  if constexpr (SL > 1) {
    __shared__ f32x4 sums[256];
    sums[threadIdx.x] = v;
    __syncthreads();
    if (slice > 0) return;
#pragma unroll
    for (int s = 1; s < SL; ++s) v += sums[s * OUT + threadIdx.x];
  }
  if (!in) return;
  v *= *scale;
  T* o = dx + i * d + e;
  if (d % 4 == 0) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else
      *reinterpret_cast<f32x4*>(o) = v;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (e + q < d) Io<T>::store(o, q, v[q]);
  }
}

// A piece's dw from the splits' sums.
template <typename T>
__global__ __launch_bounds__(256) void head_dw_out_kernel(const float* __restrict__ part, int64_t cols, int64_t d,
                                                          int64_t dp, int splits, const float* __restrict__ scale,
                                                          T* __restrict__ dw) {
  const int64_t per = (d + 3) / 4, at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= cols * per) return;
  const int64_t v = at / per, e = (at - v * per) * 4;
  f32x4 a = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) a += *reinterpret_cast<const f32x4*>(part + (s * cols + v) * dp + e);
  a *= *scale;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (e + q < d) Io<T>::store(dw, v * d + e + q, a[q]);
}

// ------------------------------------------------------------------ planning

enum What { FWD = 0, BWD = 1, STEP = 2 };

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t tiles_of(int64_t v, int64_t tile) { return (v + tile - 1) / tile; }

struct HeadPlan {
  int64_t d, dp, np, planes;
  int fold;                    // bf16, few rows: rows of one of g's two parts
  bool few;                    // bf16, few rows: head_rows_kernel copies them
  bool copy_w;                 // the head is copied (fp32, or rows that are no whole pieces)
  bool direct;                 // fp32, few rows: dx and dw by head_launch_few
  HeadShape shape, products;   // of the logits, and of dx and dw
  int64_t tiles;               // of words, forward
  int64_t vp, pieces;          // words of a piece
  int dx_splits, dw_splits;
  int64_t dx_chunk, dx_rows;
  // byte offsets in the workspace
  bool keep;                   // a step of few rows keeps their logits
  size_t rows, x, w, part, z_label, stats, factors, taught, g, z, dx, dw, total;
};

// When `slots` places that take `first` tiles of length a, then `more` of length b, are done.
double done_at(int64_t slots, int64_t first, double a, int64_t more, double b) {
  const int64_t rounds = first / slots, late = first % slots;
  // `late` places are free at (rounds + 1) a, the others at rounds a: count what fits until t, and raise t
  const double early_at = rounds * a, late_at = early_at + a;
  double t = early_at;
  for (;;) {
    const double e = floor((t - early_at) / b + 1e-9), l = t >= late_at ? floor((t - late_at) / b + 1e-9) : 0.0;
    if ((slots - late) * e + late * l >= static_cast<double>(more)) break;
    const double next_e = early_at + (e + 1) * b, next_l = t >= late_at ? late_at + (l + 1) * b : late_at + b;
    t = late > 0 && next_l < next_e ? next_l : next_e;
  }
  return late > 0 && t < late_at ? late_at : t;
}

HeadPlan head_plan(int what, int64_t rows, int64_t d, int64_t vocab, int64_t top, bool bf16) {
  HeadPlan p = {};
  p.d = d, p.dp = up(d, kPipeK), p.np = up(rows, kHeadRows), p.planes = bf16 ? 1 : 3;
  p.fold = !bf16 || rows > 64 ? 0 : rows <= kThinRows ? static_cast<int>(kThinRows) : 64;
  p.few = bf16 && rows <= kThinRows && d <= 4096;   // one workgroup's copy
  p.copy_w = !bf16 || d % 8 != 0;
  // Rounds of 256 x 256 tiles (one a CU) against rounds of 128 x 128 tiles (two a CU), which take 0.6 of the
  // time: measured, 4096 x 768 x 50257 bf16 1368 us with the first and 1456 with the second (13 and 25
  // rounds), 600 x 2000 x 10000 204 and 170 (1 and 1).
  auto rounds = [&](int64_t tile, int64_t places) { return up(tiles_of(vocab, tile) * tiles_of(rows, tile), places) / places; };
  // fp32 rows of the head that start off 16 bytes take HEAD_32's tiles, of a copy
  p.shape = rows <= kThinRows ? (bf16 || d % 4 == 0 ? HEAD_THIN : HEAD_32) : rounds(256, 256) <= 0.6 * rounds(128, 512) ? HEAD_256 : HEAD_128;
  const int64_t tv = head_tile_words(p.shape, vocab);
  p.tiles = (vocab + tv - 1) / tv;
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at = static_cast<size_t>(up(static_cast<int64_t>(at) + bytes, 256));
    return here;
  };
  p.rows = take(256 + (p.np * 3 + rows * 2) * 4);
  p.x = take(p.planes * p.np * p.dp * 2);
  p.copy_w = p.copy_w && (bf16 || p.shape != HEAD_THIN);   // which takes an fp32 head as it is
  p.w = p.copy_w ? take(p.planes * (vocab + kPipeK) * p.dp * 2) : 0;   // zeros behind: whole K tiles of words
  if (what != BWD) {
    p.part = take(p.tiles * 3 * p.np * 4);
    p.z_label = take(p.np * 4);
  }
  if (what == STEP) p.stats = take(rows * (4 + top) * 4);
  if (what != FWD) {
    p.direct = !bf16 && rows <= kThinRows;
    // np rows of each plane, but few rows hold half of that at most (as below)
    int64_t vp = up((p.fold || p.direct ? 2 : 1) * kPieceBytes / (p.planes * p.np * 2), kHeadRows) - kHeadRows;
    if (vp < kHeadRows) vp = kHeadRows;
    p.pieces = (vocab + vp - 1) / vp;
    p.vp = up((vocab + p.pieces - 1) / p.pieces, kHeadRows);
    p.pieces = (vocab + p.vp - 1) / p.vp;
    // dx: rows x features, summed over the piece's words; dw: words x features, summed over rows
    // 256 x 256 tiles where there is enough to do: 4096 x 768 x 50257 bf16 1368 us, 1494 with 128 x 128
    // (fp32 5370, 5999); 1000 x 625 x 10000 fp32 365 us, with 128 x 128 330
    const bool wide = rows > 128 && d > 128 && static_cast<double>(rows) * vocab * d >= 2e10;
    p.products = rows <= 32 ? HEAD_32 : wide ? HEAD_256 : HEAD_128;
    const int64_t xm = head_tile_features(p.products), xn = p.fold ? 128 : head_tile_rows(p.products);   // one tile of few rows
    const int64_t wm = wide ? 256 : 128;
    const int64_t slots = wide ? 256 : 512;
    const int64_t dx_tiles = tiles_of(d, xm) * tiles_of(rows, xn), dw_tiles = tiles_of(d, wm) * tiles_of(p.vp, wm);
    // dw is split only where its tiles do not fill half the chip
    int64_t ws = dw_tiles >= slots / 2 ? 1 : slots / dw_tiles;
    if (ws > (rows + 511) / 512) ws = (rows + 511) / 512;
    while (ws > 1 && ws * p.vp * p.dp * 4 > (int64_t(1) << 30)) --ws;
    p.dw_splits = static_cast<int>(ws);
    // dx's splits fill the places that dw leaves free: the split whose tiles are done first, by a tile's
    // time at the matrix instructions' rate (13 ns a k of a 256 x 256 tile, 7 of a 128 x 128 one, where two
    // share a CU; fp32 six times that) with 300 k for its start and end, and the splits' sums, written and
    // read at 2.5 TB/s (with the times that tiles take in practice, up to twice as long, splits
    // come out finer and the step slower: 1024 x 768 x 50257 bf16 400 -> 440 us)
    const double ns = (wide ? 13.0 : 7.0) * (bf16 ? 1 : 6), ends = 300.0 / (bf16 ? 1 : 6);
    double best = 0.0;
    int64_t xs = 0;
    for (int64_t n = 1; n <= 64 && (n == 1 || (p.vp / n >= 512 && n * p.np * p.dp * 4 <= (int64_t(1) << 30))); ++n) {
      const double t = ns * done_at(slots, dw_tiles * ws, static_cast<double>(rows) / ws + ends, dx_tiles * n,
                                    static_cast<double>(p.vp) / n + ends) + n * static_cast<double>(p.np * p.dp) * 4 / 2500.0;
      if (xs == 0 || t < best) best = t, xs = n;
    }
    p.dx_chunk = p.direct ? head_few_run(rows, d, p.vp) : up((p.vp + xs - 1) / xs, kPipeK);
    p.dx_splits = static_cast<int>((p.vp + p.dx_chunk - 1) / p.dx_chunk);
    p.dx_rows = p.direct ? head_few_rows(rows) : p.np;
    if (p.direct) p.dw_splits = 1;
    p.factors = take(p.np * static_cast<int64_t>(sizeof(HeadRow)));
    p.taught = take(p.np * 4);
    p.g = take(p.direct ? kThinRows * p.vp * 4 : p.fold ? 2 * p.fold * p.vp * 2 : p.planes * p.np * p.vp * 2);
    p.keep = what == STEP && p.shape == HEAD_THIN && p.pieces == 1;
    p.z = p.keep ? take(kThinRows * p.vp * 4) : 0;
    p.dx = take(p.dx_splits * p.dx_rows * p.dp * 4);
    p.dw = p.dw_splits > 1 ? take(p.dw_splits * p.vp * p.dp * 4) : 0;
  }
  p.total = at;
  return p;
}

int check_sizes(int64_t rows, int64_t d, int64_t vocab, int64_t ldx, int64_t top, int dtype) {
  if (dtype != MONARCH_F32 && dtype != MONARCH_BF16) return MONARCH_ERR_DTYPE;
  if (rows < 0 || rows >= kLimit - kHeadRows || d <= 0 || d > kMaxFeatures || vocab <= 0 || vocab > (int64_t(1) << 30) ||
      ldx < d || top < 0 || top > MONARCH_DISTILL_MAX_TOP)
    return MONARCH_ERR_SHAPE;
  return MONARCH_OK;
}

bool off_elements(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }

#define HEAD_TRY(e)                        \
  do {                                     \
    const int head_st = record_hip(e);     \
    if (head_st) return head_st;           \
  } while (0)

template <typename T>
hipError_t copy_rows(const void* src, int64_t ld, const int* idx, const int* count, int fold, int64_t rows, int64_t grid, int64_t d,
                     int64_t dp, void* dst, int64_t plane, hipStream_t s) {
  return launch_groups(grid, [&](int64_t first, dim3 g) {
    hipLaunchKernelGGL(head_copy_kernel<T>, g, dim3(256), 0, s, static_cast<const T*>(src), ld, idx, count, fold, rows, d, dp,
                       static_cast<uint16_t*>(dst), plane, first);
  });
}

template <typename T>
hipError_t dx_out(const Call& c, const HeadPlan& p, const float* part, const Rows& r, hipStream_t s) {
  const int64_t n = c.rows * ((p.d + 3) / 4);
  // 128 threads for few columns of many splits: step of 1 x 768 x 50257 fp32 156 -> 146 us, but 32 rows 236 -> 252
  const int sl = p.dx_splits >= 256 && n <= 2048 ? 128 : p.dx_splits >= 16 ? 16 : 1;
  auto kernel = sl == 128 ? head_dx_out_kernel<T, 128> : sl == 16 ? head_dx_out_kernel<T, 16> : head_dx_out_kernel<T, 1>;
  return launch_groups(tiles_of(n, 256 / sl), [&](int64_t first, dim3 g) {
    hipLaunchKernelGGL(kernel, g, dim3(256), 0, s, part, r.pos, c.rows, p.dx_rows, p.d, p.dp, p.dx_splits, r.fold, r.scale,
                       static_cast<T*>(c.dx), first);
  });
}

// One call of the three: checks are done.
int run(const Call& c, const HeadPlan& p, int what, char* ws, hipStream_t s) {
  Rows r;
  uint32_t* head = reinterpret_cast<uint32_t*>(ws + p.rows);   // 16 bytes of zeros, the count
  r.count = reinterpret_cast<int*>(head + 4);
  r.scale = reinterpret_cast<float*>(head + 5);
  r.g_rows = reinterpret_cast<int*>(head + 6);
  r.fold = p.fold;
  r.idx = reinterpret_cast<int*>(head + 64);
  r.label = r.idx + p.np;
  r.has = r.label + p.np;
  r.pos = r.has + p.np;
  r.flag = r.pos + c.rows;
  uint16_t* xc = reinterpret_cast<uint16_t*>(ws + p.x);
  if (c.taught)
    HEAD_TRY(launch_groups(tiles_of(c.rows, 4), [&](int64_t first, dim3 g) {
      hipLaunchKernelGGL(head_flag_kernel, g, dim3(256), 0, s, c, r, first);
    }));
  hipLaunchKernelGGL(head_rows_kernel, dim3(1), dim3(1024), 0, s, c, r, head, p.few ? xc : nullptr, p.dp);
  HEAD_TRY(hipGetLastError());
  const int64_t xplane = p.np * p.dp, wplane = (c.vocab + kPipeK) * p.dp;
  if (!p.few)
    HEAD_TRY(c.bf16 ? copy_rows<uint16_t>(c.x, c.ldx, r.idx, r.count, r.fold, c.rows, p.np, p.d, p.dp, xc, xplane, s)
                  : copy_rows<float>(c.x, c.ldx, r.idx, r.count, r.fold, c.rows, p.np, p.d, p.dp, xc, xplane, s));
  const uint16_t* w = static_cast<const uint16_t*>(c.w);
  int64_t ldw = p.d;
  if (p.copy_w) {
    HEAD_TRY(c.bf16 ? copy_rows<uint16_t>(c.w, p.d, nullptr, nullptr, 0, c.vocab, c.vocab + kPipeK, p.d, p.dp, ws + p.w, wplane, s)
                    : copy_rows<float>(c.w, p.d, nullptr, nullptr, 0, c.vocab, c.vocab + kPipeK, p.d, p.dp, ws + p.w, wplane, s));
    w = reinterpret_cast<const uint16_t*>(ws + p.w);
    ldw = p.dp;
  }
  HeadLogits l = {};
  l.pr.zeros = reinterpret_cast<const uint16_t*>(head);
  l.f32 = !c.bf16, l.raw = static_cast<const float*>(c.w);
  l.pr.a.p = w, l.pr.a.ld = ldw, l.pr.a.plane = wplane, l.pr.a.rows = c.vocab, l.pr.a.kvalid = ldw;   // in place the last K tile may be cut
  l.pr.b.p = xc, l.pr.b.ld = p.dp, l.pr.b.plane = xplane, l.pr.b.rows = p.np, l.pr.b.kvalid = p.dp;
  l.count = r.count, l.vocab = c.vocab, l.d = p.d, l.rows = c.rows, l.np = p.np, l.ct = kLog2e / c.temperature, l.label = r.label;
  HeadRow* factors = what == FWD ? nullptr : reinterpret_cast<HeadRow*>(ws + p.factors);
  float* taught = what == FWD ? nullptr : reinterpret_cast<float*>(ws + p.taught);
  if (what != BWD) {
    if (c.taught)
      HEAD_TRY(launch_groups(c.rows, [&](int64_t first, dim3 g) {
        if (c.bf16)
          hipLaunchKernelGGL(head_entries_kernel<uint16_t>, g, dim3(256), 0, s, c, r, static_cast<const uint16_t*>(xc), p.dp, false,
                             w, ldw, first);
        else
          hipLaunchKernelGGL(head_entries_kernel<float>, g, dim3(256), 0, s, c, r, static_cast<const float*>(c.x), c.ldx, true,
                             static_cast<const float*>(c.w), p.d, first);
      }));
    l.v0 = 0, l.v1 = c.vocab;
    l.z = p.keep ? reinterpret_cast<float*>(ws + p.z) : nullptr, l.vp = p.vp;
    l.part = reinterpret_cast<float*>(ws + p.part), l.z_label = reinterpret_cast<float*>(ws + p.z_label);
    HEAD_TRY(head_launch_sums(l, p.shape, c.second, s));
    // rows a workgroup: few are spread over the chip, many share a line's reads (with 4 and 16: 1024 x 768 x
    // 50257 6.6 and 11.7 us, 4096 rows with 64 entries 18.0 and 15.4)
    const int rw = c.rows <= 256 ? 1 : c.rows <= 2048 ? 4 : 16;
    auto loss = rw == 1 ? head_loss_kernel<1> : rw == 4 ? head_loss_kernel<4> : head_loss_kernel<16>;
    HEAD_TRY(launch_groups(p.np / rw, [&](int64_t first, dim3 g) {
      hipLaunchKernelGGL(loss, g, dim3(256), 0, s, c, r, l.part, p.np, static_cast<int>(p.tiles), l.z_label, factors, taught, first);
    }));
  }
  if (what == FWD) return MONARCH_OK;
  if (what == BWD) {
    hipLaunchKernelGGL(head_factors_kernel, dim3(static_cast<unsigned>(p.np / 256)), dim3(256), 0, s, c, r, factors, taught);
    HEAD_TRY(hipGetLastError());
  }
  uint16_t* g = reinterpret_cast<uint16_t*>(ws + p.g);
  float* gf = p.direct ? reinterpret_cast<float*>(ws + p.g) : nullptr;
  l.row = factors, l.g = g, l.few = gf, l.vp = p.vp, l.g_plane = (p.fold ? p.fold : p.np) * p.vp, l.fold = p.fold;
  HeadDx x = {};
  x.pr.zeros = l.pr.zeros, x.f32 = l.f32;
  x.pr.b.p = g, x.pr.b.ld = p.vp, x.pr.b.plane = l.g_plane, x.pr.b.rows = p.np;
  x.count = r.g_rows, x.d = p.d, x.dp = p.dp, x.np = p.np, x.chunk = p.dx_chunk, x.splits = p.dx_splits;
  x.part = reinterpret_cast<float*>(ws + p.dx);
  HeadDw y = {};
  y.pr.zeros = l.pr.zeros, y.f32 = l.f32, y.scale = r.scale;
  y.pr.a.p = xc, y.pr.a.ld = p.dp, y.pr.a.plane = xplane, y.pr.a.rows = p.dp, y.pr.a.kvalid = p.np;
  y.pr.b.p = g, y.pr.b.ld = p.vp, y.pr.b.plane = l.g_plane, y.pr.b.rows = p.vp, y.pr.b.kvalid = p.np;
  y.count = r.g_rows, y.d = p.d, y.dp = p.dp, y.splits = p.dw_splits;
  y.part = p.dw_splits > 1 ? reinterpret_cast<float*>(ws + p.dw) : nullptr;
  const int64_t es = c.bf16 ? 2 : 4;
  for (int64_t v0 = 0; v0 < c.vocab; v0 += p.vp) {
    const int64_t v1 = v0 + p.vp < c.vocab ? v0 + p.vp : c.vocab;
    l.v0 = v0, l.v1 = v1;
    if (p.keep) {
      hipLaunchKernelGGL(head_few_kernel, dim3(static_cast<unsigned>((p.vp / 4 + 255) / 256), kThinRows), dim3(256), 0, s, c, r, factors, l.z,
                         g, gf, p.vp, l.g_plane);
      HEAD_TRY(hipGetLastError());
    } else {
      HEAD_TRY(head_launch_grad(l, p.shape, c.second, s));
    }
    if (c.taught)
      HEAD_TRY(launch_groups(c.rows, [&](int64_t first, dim3 grid) {
        hipLaunchKernelGGL(head_taught_kernel, grid, dim3(64), static_cast<size_t>(c.top) * 8, s, c, r, factors, taught, g, gf, p.vp,
                           l.g_plane, p.fold ? 2 : static_cast<int>(p.planes), v0, v1, first);
      }));
    if (p.direct) {
      HeadFew f = {};
      f.g = gf, f.vp = p.vp, f.x = static_cast<const float*>(c.x), f.ldx = c.ldx, f.idx = r.idx, f.count = r.count;
      f.w = static_cast<const float*>(c.w) + v0 * p.d, f.dw = static_cast<float*>(c.dw) + v0 * p.d, f.part = x.part;
      f.d = p.d, f.dp = p.dp, f.words = v1 - v0, f.add = v0 > 0;
      HEAD_TRY(head_launch_few(f, c.rows, p.dx_chunk, p.dx_splits, s));
      continue;
    }
    x.k = up(v1 - v0, kPipeK);
    x.pr.a.p = w + v0 * ldw, x.pr.a.ld = ldw, x.pr.a.plane = wplane, x.pr.a.rows = ldw, x.pr.a.kvalid = p.copy_w ? x.k : v1 - v0;
    x.add = v0 > 0;
    y.cols = v1 - v0;
    y.dw = static_cast<char*>(c.dw) + v0 * p.d * es;
    HEAD_TRY(head_launch_products(x, y, p.products, s));
    if (y.part) {
      const unsigned n = static_cast<unsigned>((y.cols * ((p.d + 3) / 4) + 255) / 256);
      if (c.bf16)
        hipLaunchKernelGGL(head_dw_out_kernel<uint16_t>, dim3(n), dim3(256), 0, s, y.part, y.cols, p.d, p.dp, p.dw_splits,
                           r.scale, static_cast<uint16_t*>(y.dw));
      else
        hipLaunchKernelGGL(head_dw_out_kernel<float>, dim3(n), dim3(256), 0, s, y.part, y.cols, p.d, p.dp, p.dw_splits,
                           r.scale, static_cast<float*>(y.dw));
      HEAD_TRY(hipGetLastError());
    }
  }
  return record_hip(c.bf16 ? dx_out<uint16_t>(c, p, x.part, r, s) : dx_out<float>(c, p, x.part, r, s));
}

int call(Call c, int what, const void* stats_in, int64_t top, float temperature, float mix, int dtype, void* workspace,
         size_t workspace_bytes, void* stream, void* const* events, int n_events) {
  int st = check_sizes(c.rows, c.d, c.vocab, c.ldx, top, dtype);
  if (st) return st;
  if (!(temperature >= 1e-6f) || !(temperature <= 1e6f) || !(mix >= 0.0f) || !(mix <= 1.0f)) return MONARCH_ERR_VALUE;
  c.bf16 = dtype == MONARCH_BF16;
  if (top == 0) mix = 0.0f;   // the cross entropy, unweighted
  c.top = static_cast<int>(top), c.mix = mix;
  c.told = c.labels && mix < 1.0f;
  c.taught = top > 0 && mix > 0.0f;
  c.temperature = c.taught ? temperature : 1.0f;
  c.second = !c.told || !c.taught || temperature == 1.0f ? HEAD_ONE : temperature == 2.0f ? HEAD_SQUARE : HEAD_OWN;
  if (c.rows > 0) {
    if (!c.x || !c.w || (top > 0 && (!c.teacher || !c.ids))) return MONARCH_ERR_NULL;
    if (what != BWD && !c.loss) return MONARCH_ERR_NULL;
    if (what == FWD && !c.stats) return MONARCH_ERR_NULL;
    if (what == BWD && (!stats_in || !c.weight)) return MONARCH_ERR_NULL;
    if (what != FWD && !c.dx) return MONARCH_ERR_NULL;
    if (!workspace) return MONARCH_ERR_NULL;
  }
  if (what != FWD && !c.dw) return MONARCH_ERR_NULL;
  if (off_elements(c.x, c.bf16 ? 2 : 4) || misaligned(c.w) || off_elements(c.teacher, 4) || off_elements(c.ids, 8) ||
      off_elements(c.labels, 8) || off_elements(c.weight, 4) || off_elements(c.loss, 4) || misaligned(c.stats) ||
      misaligned(stats_in) || misaligned(c.dx) || misaligned(c.dw) || misaligned(workspace))
    return MONARCH_ERR_ALIGN;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (c.rows == 0) {
    if (what == FWD) return MONARCH_OK;
    return record_hip(launch_zero(c.dw, static_cast<size_t>(c.vocab * c.d) * (c.bf16 ? 2 : 4), s));
  }
  const HeadPlan p = head_plan(what, c.rows, c.d, c.vocab, top, c.bf16);
  if (workspace_bytes < p.total) return MONARCH_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  if (what == STEP) c.stats = reinterpret_cast<float*>(ws + p.stats);
  if (what == BWD) c.stats = const_cast<float*>(static_cast<const float*>(stats_in)), c.loss = nullptr;
  Tracer tr{events, n_events, 0, s};
  st = record_hip(tr.mark());
  if (st) return st;
  st = run(c, p, what, ws, s);
  if (st) return st;
  return record_hip(tr.mark());
}

}  // namespace
}  // namespace monarch

using namespace monarch;

extern "C" {

size_t monarch_head_workspace_bytes(int call, int64_t rows, int64_t features, int64_t vocab, int64_t top, int dtype) {
  if (call < 0 || call > 2 || check_sizes(rows, features, vocab, features, top, dtype) || rows == 0) return 0;
  return head_plan(call, rows, features, vocab, top, dtype == MONARCH_BF16).total;
}

size_t monarch_head_stats_bytes(int64_t rows, int64_t top) {
  if (rows < 0 || rows >= kLimit - kHeadRows || top < 0 || top > MONARCH_DISTILL_MAX_TOP) return 0;
  return static_cast<size_t>(rows) * (4 + top) * sizeof(float);
}

int monarch_head_describe(int call, int64_t rows, int64_t features, int64_t vocab, int64_t top, int dtype, char* buf,
                          size_t buf_len) {
  const int st = check_sizes(rows, features, vocab, features, top, dtype);
  if (st) return st;
  if (call < 0 || call > 2) return MONARCH_ERR_DTYPE;
  static const char* const zero = "zero_dw";
  if (rows == 0) return write_names(&zero, call == FWD ? 0 : 1, buf, buf_len);
  const HeadPlan p = head_plan(call, rows, features, vocab, top, dtype == MONARCH_BF16);
  static const char* const tile[] = {"_256", "_128", "_32", ""};   // by HeadShape
  char text[16][48];
  const char* names[16];
  int n = 0;
  auto add = [&](const char* name, const char* of, int64_t pieces) {
    if (pieces > 1)
      snprintf(text[n], sizeof text[n], "%s%s*%lld", name, of, static_cast<long long>(pieces));
    else
      snprintf(text[n], sizeof text[n], "%s%s", name, of);
    names[n] = text[n];
    ++n;
  };
  const char* logits = p.shape == HEAD_THIN ? "head_thin" : "head_sums";
  const char* again = p.shape == HEAD_THIN ? "head_thin_grad" : "head_grad";
  if (top > 0) add("head_flag", "", 1);
  add("head_rows", "", 1);
  if (!p.few) add("head_copy_x", "", 1);
  if (p.copy_w) add("head_copy_w", "", 1);
  if (call != BWD) {
    if (top > 0) add("head_entries", "", 1);
    add(logits, tile[p.shape], 1);
    add("head_loss", "", 1);
  }
  if (call != FWD) {
    if (call == BWD) add("head_factors", "", 1);
    if (p.keep)
      add("head_few", "", 1);
    else
      add(again, tile[p.shape], p.pieces);
    if (top > 0) add("head_taught", "", p.pieces);
    if (p.direct)
      add("head_few_products", "", p.pieces);
    else
      add("head_products", tile[p.products], p.pieces);
    if (p.dw_splits > 1) add("head_dw_out", "", p.pieces);
    add("head_dx_out", "", 1);
  }
  return write_names(names, n, buf, buf_len);
}

int monarch_head_fwd(const void* x, int64_t ldx, const void* w, const void* labels, const void* teacher, const void* ids,
                     void* loss, void* stats, void* workspace, size_t workspace_bytes, int64_t rows, int64_t features,
                     int64_t vocab, int64_t top, float temperature, float mix, int dtype, void* stream, void* const* events,
                     int n_events) {
  Call c = {};
  c.x = x, c.ldx = ldx, c.w = w, c.labels = static_cast<const int64_t*>(labels);
  c.teacher = static_cast<const float*>(teacher), c.ids = static_cast<const int64_t*>(ids);
  c.loss = static_cast<float*>(loss), c.stats = static_cast<float*>(stats);
  c.rows = rows, c.d = features, c.vocab = vocab;
  return call(c, FWD, nullptr, top, temperature, mix, dtype, workspace, workspace_bytes, stream, events, n_events);
}

int monarch_head_bwd(const void* dloss, const void* x, int64_t ldx, const void* w, const void* labels, const void* teacher,
                     const void* ids, const void* stats, void* dx, void* dw, void* workspace, size_t workspace_bytes,
                     int64_t rows, int64_t features, int64_t vocab, int64_t top, float temperature, float mix, int dtype,
                     void* stream, void* const* events, int n_events) {
  Call c = {};
  c.x = x, c.ldx = ldx, c.w = w, c.labels = static_cast<const int64_t*>(labels);
  c.teacher = static_cast<const float*>(teacher), c.ids = static_cast<const int64_t*>(ids);
  c.weight = static_cast<const float*>(dloss), c.dx = dx, c.dw = dw;
  c.rows = rows, c.d = features, c.vocab = vocab;
  return call(c, BWD, stats, top, temperature, mix, dtype, workspace, workspace_bytes, stream, events, n_events);
}

int monarch_head_step(const void* x, int64_t ldx, const void* w, const void* labels, const void* teacher, const void* ids,
                      const void* row_weight, void* loss, void* dx, void* dw, void* workspace, size_t workspace_bytes,
                      int64_t rows, int64_t features, int64_t vocab, int64_t top, float temperature, float mix, int dtype,
                      void* stream, void* const* events, int n_events) {
  Call c = {};
  c.x = x, c.ldx = ldx, c.w = w, c.labels = static_cast<const int64_t*>(labels);
  c.teacher = static_cast<const float*>(teacher), c.ids = static_cast<const int64_t*>(ids);
  c.weight = static_cast<const float*>(row_weight), c.loss = static_cast<float*>(loss), c.dx = dx, c.dw = dw;
  c.rows = rows, c.d = features, c.vocab = vocab;
  return call(c, STEP, nullptr, top, temperature, mix, dtype, workspace, workspace_bytes, stream, events, n_events);
}

}  // extern "C"
