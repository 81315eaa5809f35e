// The three products of the head loss, each with its epilogue (gfx950).
//
//   logits   z[v, n] = sum_d w[v, d] x[n, d]     words down, rows across: a lane holds
//            4 consecutive words of one row in each MFMA tile, so that a row's
//            maximum and sum of exponentials are taken in registers, four lanes
//            meet by two swaps, and only (maximum, sums) of a tile leave the chip;
//            or, for the gradient, g = a q + b s - off [v = label], rounded to
//            bf16 (up to 64 rows two bf16 parts; fp32: three, exact), [n][v] through LDS.
//   dx       [d, n] = sum_v w[v, d] g[n, v]       split over the words
//   dw       [d, v] = sum_n x[n, d] g[n, v]
//
// g is one piece of the vocabulary, in the workspace: at most 1 GiB, or 256 words of it.
#include "head.h"
#include "kernels.h"

namespace monarch {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLowest = -3.402823466e38f;

using Shape256 = PipeShape<2, 4, 8, 4, 2>;
using Shape128 = PipeShape<2, 2, 4, 4, 2>;
using Shape32 = PipeShape<4, 1, 2, 2, 4>;
using Shape64 = PipeShape<4, 1, 2, 4, 3>;   // dx of few rows

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// Workgroup b of a grid: consecutive tiles share an XCD (workgroups are dealt round
// to the 8 of them), and with it an L2.
__device__ __forceinline__ int64_t xcd_tile(int64_t b, int64_t n) {
  const int64_t x = b & 7, i = b >> 3, per = n >> 3, more = n & 7;
  return x * per + (x < more ? x : more) + i;
}

// max / sum over the four lanes that hold one column of MFMA tiles (lane % 16 alike)
template <bool MAX>
__device__ __forceinline__ float over_groups(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
  v = MAX ? fmaxf(a, b) : a + b;
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
  return MAX ? fmaxf(a, b) : a + b;
}

// Tile t of an outer x inner grid of tiles: the inner ones in panels of 8, a panel's outer ones
// after each other, so that the 32 workgroups that an XCD runs together take about 4 x 8 tiles
// and share their operands' tiles in its L2 (12 of 64 K tiles come from outside it; 18 where 16 x 2
// run together).
__device__ __forceinline__ void panel_tile(int64_t t, int64_t outer, int64_t inner, int64_t* o, int64_t* i) {
  const int64_t panel = t / (8 * outer), wide = inner - panel * 8 < 8 ? inner - panel * 8 : 8;
  const int64_t r = t - panel * 8 * outer;
  *o = r / wide;
  *i = panel * 8 + r % wide;
}

template <class S, HeadSecond SECOND, bool F32>
__global__ __launch_bounds__(S::NT) void head_sums_kernel(HeadLogits p, int64_t vt, int64_t nt, int64_t group) {
  __shared__ __attribute__((aligned(16))) char lds[S::LDS];
  int64_t tv, tn;
  panel_tile(group + xcd_tile(blockIdx.x, gridDim.x), vt, nt, &tv, &tn);
  const int64_t v0 = p.v0 + tv * S::BM, n0 = tn * S::BN;
  if (n0 >= *p.count) return;
  f32x4 acc[S::FM][S::FN];
  pipe_clear<S>(acc);
  pipe_product<S, false, false, F32>(p.pr, v0, n0, 0, p.d, lds, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / S::WN, wn = wave % S::WN, l15 = lane & 15, lh = lane >> 4;
  const int64_t vw = v0 + wm * S::FM * 16 + 4 * lh;   // this lane's first word
  const bool cut = v0 + S::BM > p.v1;
  float* part = reinterpret_cast<float*>(lds);        // [WM][3][BN]
#pragma unroll
  for (int ni = 0; ni < S::FN; ++ni) {
    const int col = (wn * S::FN + ni) * 16 + l15;
    if (cut) {
#pragma unroll
      for (int mi = 0; mi < S::FM; ++mi)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (vw + mi * 16 + v >= p.v1) acc[mi][ni][v] = -INFINITY;
    }
    float m = kLowest;
#pragma unroll
    for (int mi = 0; mi < S::FM; ++mi)
      m = fmaxf(fmaxf(fmaxf(m, acc[mi][ni][0]), fmaxf(acc[mi][ni][1], acc[mi][ni][2])), acc[mi][ni][3]);
    m = over_groups<true>(m);
    float st = 0.f, s1 = 0.f;
#pragma unroll
    for (int mi = 0; mi < S::FM; ++mi)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float z = acc[mi][ni][v] - m;
        const float e = exp2_of(z * p.ct);
        st += e;
        if constexpr (SECOND == HEAD_OWN) s1 += exp2_of(z * kLog2e);
        if constexpr (SECOND == HEAD_SQUARE) s1 = fmaf(e, e, s1);
      }
    st = over_groups<false>(st);
    if constexpr (SECOND != HEAD_ONE) s1 = over_groups<false>(s1);
    if (lh == 0) {
      part[(wm * 3 + 0) * S::BN + col] = m;
      part[(wm * 3 + 1) * S::BN + col] = st;
      part[(wm * 3 + 2) * S::BN + col] = SECOND != HEAD_ONE ? s1 : 0.f;
    }
    // the lane that holds the label's logit hands it out
    const int64_t at = static_cast<int64_t>(p.label[n0 + col]) - vw;
    const bool mine = at >= 0 && at < S::FM * 16 && (at & 15) < 4;
    if (__any(mine)) {
#pragma unroll
      for (int mi = 0; mi < S::FM; ++mi)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (at == mi * 16 + v) p.z_label[n0 + col] = acc[mi][ni][v];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < S::BN; c += S::NT) {
    float m = part[c];
#pragma unroll
    for (int w = 1; w < S::WM; ++w) m = fmaxf(m, part[w * 3 * S::BN + c]);
    float st = 0.f, s1 = 0.f;
#pragma unroll
    for (int w = 0; w < S::WM; ++w) {
      const float by = part[w * 3 * S::BN + c] - m;
      st += part[(w * 3 + 1) * S::BN + c] * exp2_of(by * p.ct);
      if constexpr (SECOND != HEAD_ONE) s1 += part[(w * 3 + 2) * S::BN + c] * exp2_of(by * kLog2e);
    }
    float* o = p.part + (tv * 3) * p.np + n0 + c;
    o[0] = m;
    o[p.np] = st;
    o[2 * p.np] = SECOND != HEAD_ONE ? s1 : st;
  }
}

// Four fp32 values as bf16.
__device__ __forceinline__ u32x2 rounded(const f32x4& v) {
  return u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// Four fp32 values as bf16, and what is left of them (the next plane's).
__device__ __forceinline__ u32x2 next_plane(f32x4& v) {
  const u32x2 r = {pack_bf16x2(finite_bf16(v[0]), finite_bf16(v[1])), pack_bf16x2(finite_bf16(v[2]), finite_bf16(v[3]))};
  const float hi[4] = {__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u),
                       __uint_as_float(r[1] << 16), __uint_as_float(r[1] & 0xffff0000u)};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = isfinite(v[i]) ? v[i] - hi[i] : 0.f;
  return r;
}

// Byte offset in LDS of 8 bytes (4 elements) at element e of row r of a bf16 tile
// with ROW elements a row: 16-byte pieces swapped within a row by r, so that the 16
// rows of a store fall on all banks.
template <int ROW>
__device__ __forceinline__ int staged(int r, int e) {
  constexpr int M = ROW / 8 < 32 ? ROW / 8 - 1 : 31;
  return r * ROW * 2 + ((((e >> 3) ^ (r & M)) << 4) | ((e & 4) << 1));
}

template <class S, HeadSecond SECOND, bool F32>
__global__ __launch_bounds__(S::NT) void head_grad_kernel(HeadLogits p, int64_t vt, int64_t nt, int64_t group) {
  static_assert(S::BM * S::BN * 2 <= S::LDS, "a tile of g is staged in LDS");
  __shared__ __attribute__((aligned(16))) char lds[S::LDS];
  int64_t tv, tn;
  panel_tile(group + xcd_tile(blockIdx.x, gridDim.x), vt, nt, &tv, &tn);
  const int64_t v0 = p.v0 + tv * S::BM, n0 = tn * S::BN;
  if (n0 >= *p.count) return;
  f32x4 acc[S::FM][S::FN];
  pipe_clear<S>(acc);
  pipe_product<S, false, false, F32>(p.pr, v0, n0, 0, p.d, lds, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / S::WN, wn = wave % S::WN, l15 = lane & 15, lh = lane >> 4;
  const int64_t vw = v0 + wm * S::FM * 16 + 4 * lh;
  const bool cut = v0 + S::BM > p.v1;
#pragma unroll
  for (int ni = 0; ni < S::FN; ++ni) {
    const int64_t n = n0 + (wn * S::FN + ni) * 16 + l15;
    const HeadRow r = p.row[n];
    const int64_t at = static_cast<int64_t>(p.label[n]) - vw;
    const bool mine = at >= 0 && at < S::FM * 16 && (at & 15) < 4;
    const bool any = __any(mine);
#pragma unroll
    for (int mi = 0; mi < S::FM; ++mi) {
      f32x4 g;
#pragma unroll
      for (int v = 0; v < 4; ++v) g[v] = head_g<SECOND>(r, acc[mi][ni][v], p.ct, false);
      if (any) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (at == mi * 16 + v) g[v] -= r.off;
      }
      if (cut) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (vw + mi * 16 + v >= p.v1) g[v] = 0.f;
      }
      acc[mi][ni] = g;
    }
  }
  if constexpr (std::is_same<S, Shape32>::value) {   // one tile of rows
#pragma unroll
    for (int ni = 0; ni < S::FN; ++ni)
#pragma unroll
      for (int mi = 0; mi < S::FM; ++mi)
        *reinterpret_cast<f32x4*>(p.few + ((wn * S::FN + ni) * 16 + l15) * p.vp + (vw - p.v0) + mi * 16) = acc[mi][ni];
    return;
  }
  const int planes = F32 ? 3 : p.fold ? 2 : 1;
  for (int k = 0; k < planes; ++k) {
    if (k > 0) __syncthreads();
#pragma unroll
    for (int ni = 0; ni < S::FN; ++ni)
#pragma unroll
      for (int mi = 0; mi < S::FM; ++mi) {
        const u32x2 w = F32 || planes > 1 ? next_plane(acc[mi][ni]) : rounded(acc[mi][ni]);
        *reinterpret_cast<u32x2*>(lds + staged<S::BM>((wn * S::FN + ni) * 16 + l15, (wm * S::FM + mi) * 16 + 4 * lh)) = w;
      }
    __syncthreads();
    constexpr int CH = S::BM / 8;
    uint16_t* out = p.g + k * p.g_plane + n0 * p.vp + tv * S::BM;
    for (int c = threadIdx.x; c < S::BN * CH; c += S::NT) {
      const int row = c / CH, e = (c % CH) * 8;
      if (!F32 && p.fold && n0 + row >= p.fold) continue;   // there the second part's rows lie
      *reinterpret_cast<u32x4*>(out + row * p.vp + e) = *reinterpret_cast<const u32x4*>(lds + staged<S::BM>(row, e));
    }
  }
}

// Logits of at most 16 * NB rows: bound by reading the head once. A workgroup takes a run of
// words, 64 at a time, 16 a wave, and a head's row comes in pieces of 512 bytes: K tiles of 256 (fp32:
// 128) go straight into LDS, three in flight, one after another over the run's words, so that
// loads never pause. A row's maximum and sums run on in registers over the run; lanes meet at its end.
// Read in pieces of 128 bytes (tiles of 128 words and 32 rows), the forward pass of 32 x 4096 x 131072 bf16 takes
// 400 us, this way 267 (4.0 TB/s). In fp32 the head is taken as it is and cut into its three bf16 parts
// in registers, where the wider tiles read a copy of planes.
//
// A K tile's row r holds its 16-byte piece q at q ^ (r mod 16): the 16 rows of a read fall on all banks.
constexpr int kThinWords = 64;

template <int NB, bool F32>
struct ThinShape {
  static constexpr int K = F32 ? 128 : 256;
  // 1 KB loads of a K tile: the words' rows of 512 bytes, then the rows' (fp32: of 256 bytes in each of three planes)
  static constexpr int W_LOADS = kThinWords / 2, LOADS = W_LOADS + (F32 ? 3 * 16 * NB / 4 : 16 * NB / 2);
  static constexpr int STAGE = LOADS * 1024, NST = F32 && NB == 2 ? 2 : 3, LDS = STAGE * NST;
  static constexpr int PER = LOADS / 4;
};

// 8 fp32 values as three bf16 fragments.
__device__ __forceinline__ void three_parts(f32x4 lo, f32x4 hi, bf16x8 (&f)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const u32x2 a = next_plane(lo), b = next_plane(hi);
    const u32x4 v = {a[0], a[1], b[0], b[1]};
    __builtin_memcpy(&f[q], &v, 16);
  }
}

template <int NB, bool GRAD, HeadSecond SECOND, bool F32>
__global__ __launch_bounds__(256) void head_thin_kernel(HeadLogits p, int64_t run) {
  using S = ThinShape<NB, F32>;
  constexpr int NST = S::NST, PER = S::PER, kThinK = S::K;
  __shared__ __attribute__((aligned(16))) char lds[S::LDS];
  __shared__ float part[4][3][16 * NB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l15 = lane & 15, lh = lane >> 4;
  const int64_t first = p.v0 + blockIdx.x * run, end = first + run < p.v1 ? first + run : p.v1;
  const int64_t kw = F32 ? p.d : p.pr.a.kvalid, kx = p.pr.b.kvalid;
  const int ktiles = static_cast<int>((kw + kThinK - 1) / kThinK);
  const int ntiles = static_cast<int>((end - first + kThinWords - 1) / kThinWords) * ktiles;
  int lk = 0;
  int64_t lv = first;
  auto issue = [&](int st) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = wave * PER + i;
      const void* s = p.pr.zeros;
      if (j < S::W_LOADS) {
        const int row = j * 2 + (lane >> 5), piece = (lane & 31) ^ (row & 15);
        const int64_t v = lv + row, k = lk * kThinK + piece * (F32 ? 4 : 8);
        if (v < end && k < kw) {
          if constexpr (F32)
            s = p.raw + v * p.d + k;
          else
            s = p.pr.a.p + v * p.pr.a.ld + k;
        }
      } else if constexpr (F32) {
        const int row = (j - S::W_LOADS) * 4 + (lane >> 4), plane = row / (16 * NB), r = row % (16 * NB);
        const int64_t k = lk * kThinK + (((lane & 15) ^ (r & 15)) << 3);
        if (k < kx) s = p.pr.b.p + plane * p.pr.b.plane + r * p.pr.b.ld + k;
      } else {
        const int row = (j - S::W_LOADS) * 2 + (lane >> 5);
        const int64_t k = lk * kThinK + (((lane & 31) ^ (row & 15)) << 3);
        if (k < kx) s = p.pr.b.p + row * p.pr.b.ld + k;
      }
      __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)(s),
                                       (__attribute__((address_space(3))) void*)(lds + st * S::STAGE + j * 1024), 16, 0, 0);
    }
    if (++lk == ktiles) lk = 0, lv += kThinWords;
  };
  f32x4 acc[NB];
  float m[NB], st[NB], s1[NB];
  int label[NB];
  HeadRow r[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    m[b] = kLowest, st[b] = 0.f, s1[b] = 0.f;
    label[b] = p.label[b * 16 + l15];
    if constexpr (GRAD) r[b] = p.row[b * 16 + l15];
  }
  for (int t = 0; t < NST && t < ntiles; ++t) issue(t);
  int k = 0, place = 0;
  int64_t v0 = first;
#pragma unroll 1
  for (int t = 0; t < ntiles; ++t) {
    const int later = ntiles - 1 - t < NST - 1 ? ntiles - 1 - t : NST - 1;
    asm volatile("" ::: "memory");
    pipe_wait_stages<PER, NST - 1>(later);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const char* at = lds + place * S::STAGE;
    const char* words = at + (wave * 16 + l15) * 512;
    const char* rows = at + S::W_LOADS * 1024;
#pragma unroll
    for (int u = 0; u < kThinK / 32; ++u) {
      if constexpr (F32) {
        const int piece = 8 * u + 2 * lh;
        bf16x8 fa[3];
        three_parts(*reinterpret_cast<const f32x4*>(words + ((piece ^ l15) << 4)),
                    *reinterpret_cast<const f32x4*>(words + (((piece + 1) ^ l15) << 4)), fa);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          bf16x8 fb[3];
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(rows + ((q * NB + b) * 16 + l15) * 256 + (((4 * u + lh) ^ l15) << 4));
            __builtin_memcpy(&fb[q], &x, 16);
          }
          constexpr int pa[6] = {2, 0, 1, 1, 0, 0}, pb[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
          for (int q = 0; q < 6; ++q) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[pa[q]], fb[pb[q]], acc[b], 0, 0, 0);
        }
      } else {
        const int piece = ((4 * u + lh) ^ l15) << 4;
        bf16x8 fa, fb;
        const u32x4 a = *reinterpret_cast<const u32x4*>(words + piece);
        __builtin_memcpy(&fa, &a, 16);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(rows + (b * 16 + l15) * 512 + piece);
          __builtin_memcpy(&fb, &x, 16);
          acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, fb, acc[b], 0, 0, 0);
        }
      }
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(pipe_wait(63));   // its reads are done
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (t + NST < ntiles) issue(place);
    place = place + 1 == NST ? 0 : place + 1;
    if (++k < ktiles) continue;
    k = 0;
    const int64_t vw = v0 + wave * 16 + 4 * lh;
    v0 += kThinWords;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int n = b * 16 + l15;
      const int64_t own = label[b] - vw;
      if constexpr (GRAD) {
        f32x4 g;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          g[v] = head_g<SECOND>(r[b], acc[b][v], p.ct, own == v);
          if (vw + v >= end) g[v] = 0.f;
        }
        // a gradient's runs are whole tiles, as K tiles of dx's are (behind the last word g has room)
        if constexpr (F32) {
          *reinterpret_cast<f32x4*>(p.few + n * p.vp + (vw - p.v0)) = g;
        } else {
          uint16_t* o = p.g + n * p.vp + (vw - p.v0);
#pragma unroll
          for (int q = 0; q < 2; ++q, o += p.g_plane) {
            *reinterpret_cast<u32x2*>(o) = next_plane(g);
            // the other rows of the part's half of a K tile of dw's are 0
            if constexpr (NB == 1) *reinterpret_cast<u32x2*>(o + 16 * p.vp) = u32x2{0, 0};
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (vw + v >= end) acc[b][v] = -INFINITY;
          if (own == v && vw + v < end) p.z_label[n] = acc[b][v];
        }
        if (p.z && vw < end) *reinterpret_cast<f32x4*>(p.z + n * p.vp + (vw - p.v0)) = acc[b];
        const float to = fmaxf(fmaxf(fmaxf(m[b], acc[b][0]), fmaxf(acc[b][1], acc[b][2])), acc[b][3]);
        st[b] *= exp2_of((m[b] - to) * p.ct);
        if constexpr (SECOND != HEAD_ONE) s1[b] *= exp2_of((m[b] - to) * kLog2e);
        m[b] = to;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float z = acc[b][v] - to, e = exp2_of(z * p.ct);
          st[b] += e;
          if constexpr (SECOND == HEAD_OWN) s1[b] += exp2_of(z * kLog2e);
          if constexpr (SECOND == HEAD_SQUARE) s1[b] = fmaf(e, e, s1[b]);
        }
      }
      acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  if constexpr (!GRAD) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float to = over_groups<true>(m[b]);
      st[b] = over_groups<false>(st[b] * exp2_of((m[b] - to) * p.ct));
      if constexpr (SECOND != HEAD_ONE) s1[b] = over_groups<false>(s1[b] * exp2_of((m[b] - to) * kLog2e));
      if (lh == 0) part[wave][0][b * 16 + l15] = to, part[wave][1][b * 16 + l15] = st[b], part[wave][2][b * 16 + l15] = s1[b];
    }
    __syncthreads();
    if (threadIdx.x < 16 * NB) {
      const int n = threadIdx.x;
      float to = part[0][0][n], t = 0.f, o1 = 0.f;
#pragma unroll
      for (int i = 1; i < 4; ++i) to = fmaxf(to, part[i][0][n]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float by = part[i][0][n] - to;
        t += part[i][1][n] * exp2_of(by * p.ct);
        if constexpr (SECOND != HEAD_ONE) o1 += part[i][2][n] * exp2_of(by * kLog2e);
      }
      float* o = p.part + static_cast<int64_t>(blockIdx.x) * 3 * p.np + n;
      o[0] = to;
      o[p.np] = t;
      o[2 * p.np] = SECOND != HEAD_ONE ? o1 : t;
    }
  }
}

template <class S, bool F32>
__device__ __forceinline__ void dx_tile(const HeadDx& p, int64_t at, char* lds) {
  const int64_t dt = p.dt, nt = p.nt;
  const int64_t t = xcd_tile(at, dt * nt * p.splits), split = t / (dt * nt);
  int64_t td, tn;
  panel_tile(t - split * dt * nt, nt, dt, &tn, &td);
  const int64_t d0 = td * S::BM, n0 = tn * S::BN;
  if (n0 >= *p.count) return;
  const int64_t kb = split * p.chunk, ke = kb + p.chunk < p.k ? kb + p.chunk : p.k;
  f32x4 acc[S::FM][S::FN];
  pipe_clear<S>(acc);
  pipe_product<S, true, false, F32>(p.pr, d0, n0, kb, ke, lds, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / S::WN, wn = wave % S::WN, l15 = lane & 15, lh = lane >> 4;
#pragma unroll
  for (int ni = 0; ni < S::FN; ++ni) {
    const int64_t n = n0 + (wn * S::FN + ni) * 16 + l15;
    float* o = p.part + (split * p.np + n) * p.dp;
#pragma unroll
    for (int mi = 0; mi < S::FM; ++mi) {
      const int64_t d = d0 + (wm * S::FM + mi) * 16 + 4 * lh;
      if (d < p.dp) {   // dp is a multiple of 64
        f32x4* at = reinterpret_cast<f32x4*>(o + d);
        *at = p.add ? acc[mi][ni] + *at : acc[mi][ni];
      }
    }
  }
}

template <class S, bool F32>
__device__ __forceinline__ void dw_tile(const HeadDw& p, int64_t at, char* lds) {
  const int64_t dt = p.dt, vt = p.vt;
  const int64_t t = xcd_tile(at, dt * vt * p.splits), split = t / (dt * vt);
  int64_t td, tv;
  panel_tile(t - split * dt * vt, vt, dt, &tv, &td);
  const int64_t d0 = td * S::BM, v0 = tv * S::BN;
  const int64_t count = *p.count;
  const int64_t steps = (count + kPipeK - 1) / kPipeK, per = (steps + p.splits - 1) / p.splits;
  const int64_t kb = split * per * kPipeK, end = (split + 1) * per < steps ? (split + 1) * per : steps;
  f32x4 acc[S::FM][S::FN];
  pipe_clear<S>(acc);
  pipe_product<S, true, true, F32>(p.pr, d0, v0, kb, end * kPipeK, lds, acc);
  if (!F32 && !p.part) {
    const float scale = *p.scale;
#pragma unroll
    for (int mi = 0; mi < S::FM; ++mi)
#pragma unroll
      for (int ni = 0; ni < S::FN; ++ni) acc[mi][ni] *= scale;
  }

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / S::WN, wn = wave % S::WN, l15 = lane & 15, lh = lane >> 4;
  if (F32 || p.part) {
    // fp32: a split's sums, or the result
    const int64_t ld = p.part ? p.dp : p.d;
    float* base = p.part ? p.part + split * p.cols * p.dp : static_cast<float*>(p.dw);
#pragma unroll
    for (int ni = 0; ni < S::FN; ++ni) {
      const int64_t v = v0 + (wn * S::FN + ni) * 16 + l15;
      if (v >= p.cols) continue;
      float* o = base + v * ld;
#pragma unroll
      for (int mi = 0; mi < S::FM; ++mi) {
        const int64_t d = d0 + (wm * S::FM + mi) * 16 + 4 * lh;
        if (ld % 4 == 0) {
          if (d < ld) *reinterpret_cast<f32x4*>(o + d) = acc[mi][ni];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (d + e < ld) o[d + e] = acc[mi][ni][e];
        }
      }
    }
    return;
  }
  static_assert(S::BM * S::BN * 2 <= S::LDS, "a tile of dw is staged in LDS");
#pragma unroll
  for (int ni = 0; ni < S::FN; ++ni)
#pragma unroll
    for (int mi = 0; mi < S::FM; ++mi) {
      const u32x2 w = {pack_bf16x2(acc[mi][ni][0], acc[mi][ni][1]), pack_bf16x2(acc[mi][ni][2], acc[mi][ni][3])};
      *reinterpret_cast<u32x2*>(lds + staged<S::BM>((wn * S::FN + ni) * 16 + l15, (wm * S::FM + mi) * 16 + 4 * lh)) = w;
    }
  __syncthreads();
  uint16_t* dw = static_cast<uint16_t*>(p.dw);
  if (p.d % 8 == 0) {
    constexpr int CH = S::BM / 8;
    for (int c = threadIdx.x; c < S::BN * CH; c += S::NT) {
      const int row = c / CH, e = (c % CH) * 8;
      if (v0 + row < p.cols && d0 + e < p.d)
        __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(lds + staged<S::BM>(row, e)),
                                    reinterpret_cast<u32x4*>(dw + (v0 + row) * p.d + d0 + e));
    }
  } else {
    for (int c = threadIdx.x; c < S::BN * S::BM; c += S::NT) {
      const int row = c / S::BM, e = c % S::BM;
      if (v0 + row < p.cols && d0 + e < p.d)
        dw[(v0 + row) * p.d + d0 + e] = *reinterpret_cast<const uint16_t*>(lds + staged<S::BM>(row, e) + (e & 3) * 2);
    }
  }
}

// Both products of a piece of g in one launch: neither fills the chip in whole rounds by
// itself, and dx's shorter tiles take the places that dw's leave free (16384 x 768 x
// 25128 words: dw alone is 1.16 rounds).
template <class SX, class SW, bool F32>
__global__ __launch_bounds__(SX::NT) void head_products_kernel(HeadDx x, HeadDw w, int64_t dw_tiles) {
  static_assert(SX::NT == SW::NT, "one workgroup size");
  __shared__ __attribute__((aligned(16))) char lds[SX::LDS > SW::LDS ? SX::LDS : SW::LDS];
  const int64_t at = blockIdx.x;
  if (at < dw_tiles)
    dw_tile<SW, F32>(w, at, lds);
  else
    dx_tile<SX, F32>(x, at - dw_tiles, lds);
}

// dx and dw of at most R rows in fp32: a wave takes 64 C columns and a run of words. Their rows of x and of dx's
// sums stay in its registers, each word's columns are read once, and written as dw's; g comes through scalar
// registers, four words of a row at a time. Bound by reading w and writing dw up to 16 rows (at
// 32 the fp32 units' rate is as near). By bf16 parts and matrix instructions the head was first copied as
// three planes and g's K tiles were mostly zeros: step of 8 x 768 x 50257 278 -> 157 us.
template <int R, int C, bool WHOLE>
__global__ __launch_bounds__(64) void head_few_products_kernel(const float* __restrict__ g, int64_t vp, const float* __restrict__ x,
                                                               int64_t ldx, const int* __restrict__ idx,
                                                               const int* __restrict__ count, const float* __restrict__ w,
                                                               float* __restrict__ dw, float* __restrict__ part, int64_t d,
                                                               int64_t dp, int64_t words, int64_t run, bool add) {
  constexpr int U = 4;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * (64 * C) + (WHOLE ? threadIdx.x * C : threadIdx.x);
  // columns c0 + i, or c0 + 64 i where rows are no whole pieces
  auto column = [&](int i) { return c0 + (WHOLE ? i : 64 * i); };
  const int64_t first = blockIdx.x * run, end = first + run < words ? first + run : words;
  const int rows = *count;
  float xs[R][C], dx[R][C];
#pragma unroll
  for (int n = 0; n < R; ++n) {
    const float* row = x + (n < rows ? idx[n] : 0) * ldx;
#pragma unroll
    for (int i = 0; i < C; ++i) xs[n][i] = n < rows && column(i) < d ? row[column(i)] : 0.f, dx[n][i] = 0.f;
  }
  auto load = [&](int64_t v, float (&o)[C]) {
    const float* at = w + v * d;
    if constexpr (WHOLE) {
      if (c0 < d) __builtin_memcpy(o, __builtin_assume_aligned(at + c0, 4 * C), 4 * C);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (column(i) < d) o[i] = at[column(i)];
    }
  };
  auto store = [&](int64_t v, const float (&o)[C]) {
    float* at = dw + v * d;
    if constexpr (WHOLE) {
      typedef float piece __attribute__((ext_vector_type(C)));
      piece q;
      __builtin_memcpy(&q, o, 4 * C);
      if (c0 < d) __builtin_nontemporal_store(q, reinterpret_cast<piece*>(at + c0));
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (column(i) < d) at[column(i)] = o[i];
    }
  };
  if (rows > 0) {
    float next[U][C] = {};
    auto fetch = [&](int64_t v) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v + u < end) load(v + u, next[u]);
    };
    fetch(first);
    for (int64_t v = first; v < end; v += U) {
      float now[U][C], s[U][C] = {};
      __builtin_memcpy(now, next, sizeof(now));
      fetch(v + U);
#pragma unroll
      for (int n = 0; n < R; ++n) {
        // behind the last word g is 0 up to vp, a multiple of 256
        const f32x4 q = *reinterpret_cast<const f32x4*>(g + n * vp + v);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < C; ++i) {
            s[u][i] = fmaf(q[u], xs[n][i], s[u][i]);
            // what lies behind the run's last word is another's
            if (u == 0 || v + u < end) dx[n][i] = fmaf(q[u], now[u][i], dx[n][i]);
          }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v + u < end) store(v + u, s[u]);
    }
  } else {
    const float none[C] = {};
    for (int64_t v = first; v < end; ++v) store(v, none);
  }
#pragma unroll
  for (int n = 0; n < R; ++n) {
    float* o = part + (blockIdx.x * static_cast<int64_t>(R) + n) * dp;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (column(i) < d) o[column(i)] = add ? o[column(i)] + dx[n][i] : dx[n][i];
  }
}

template <int R, int C>
hipError_t few(const HeadFew& a, int64_t run, int64_t splits, hipStream_t st) {
  const int64_t cols = (a.d + 64 * C - 1) / (64 * C);
  auto kernel = a.d % 4 == 0 ? head_few_products_kernel<R, C, true> : head_few_products_kernel<R, C, false>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(splits), static_cast<unsigned>(cols)), dim3(64), 0, st, a.g, a.vp, a.x,
                     a.ldx, a.idx, a.count, a.w, a.dw, a.part, a.d, a.dp, a.words, run, a.add);
  return hipGetLastError();
}

int64_t tiles(int64_t n, int64_t by) { return (n + by - 1) / by; }

template <class S, bool GRAD, HeadSecond SECOND, bool F32>
hipError_t logits(const HeadLogits& a, hipStream_t st) {
  const int64_t vt = tiles(a.v1 - a.v0, S::BM), nt = tiles(a.np, S::BN);
  return launch_groups(vt * nt, [&](int64_t first, dim3 g) {
    if constexpr (GRAD)
      hipLaunchKernelGGL((head_grad_kernel<S, SECOND, F32>), g, dim3(S::NT), 0, st, a, vt, nt, first);
    else
      hipLaunchKernelGGL((head_sums_kernel<S, SECOND, F32>), g, dim3(S::NT), 0, st, a, vt, nt, first);
  });
}

template <class S, bool GRAD>
hipError_t logits(const HeadLogits& a, HeadSecond second, hipStream_t st) {
  if (second == HEAD_ONE) return a.f32 ? logits<S, GRAD, HEAD_ONE, true>(a, st) : logits<S, GRAD, HEAD_ONE, false>(a, st);
  if (second == HEAD_OWN) return a.f32 ? logits<S, GRAD, HEAD_OWN, true>(a, st) : logits<S, GRAD, HEAD_OWN, false>(a, st);
  return a.f32 ? logits<S, GRAD, HEAD_SQUARE, true>(a, st) : logits<S, GRAD, HEAD_SQUARE, false>(a, st);
}

// Words of a workgroup's run, for one workgroup a CU: whole tiles, or whole waves' words.
int64_t thin_run(int64_t words, int64_t of) { return tiles(words, 256 * of) * of; }

template <bool GRAD, int NB, bool F32>
hipError_t thin(const HeadLogits& a, HeadSecond second, hipStream_t st) {
  const int64_t run = thin_run(a.v1 - a.v0, GRAD ? kThinWords : 16);
  const dim3 g(static_cast<unsigned>(tiles(a.v1 - a.v0, run)));
  if (second == HEAD_ONE)
    hipLaunchKernelGGL((head_thin_kernel<NB, GRAD, HEAD_ONE, F32>), g, dim3(256), 0, st, a, run);
  else if (second == HEAD_OWN)
    hipLaunchKernelGGL((head_thin_kernel<NB, GRAD, HEAD_OWN, F32>), g, dim3(256), 0, st, a, run);
  else
    hipLaunchKernelGGL((head_thin_kernel<NB, GRAD, HEAD_SQUARE, F32>), g, dim3(256), 0, st, a, run);
  return hipGetLastError();
}

template <bool GRAD>
hipError_t logits(const HeadLogits& a, HeadShape s, HeadSecond second, hipStream_t st) {
  if (s == HEAD_THIN) {
    if (a.f32) return a.rows <= 16 ? thin<GRAD, 1, true>(a, second, st) : thin<GRAD, 2, true>(a, second, st);
    return a.rows <= 16 ? thin<GRAD, 1, false>(a, second, st) : thin<GRAD, 2, false>(a, second, st);
  }
  if (s == HEAD_32)
    return second == HEAD_ONE   ? logits<Shape32, GRAD, HEAD_ONE, true>(a, st)
           : second == HEAD_OWN ? logits<Shape32, GRAD, HEAD_OWN, true>(a, st)
                                : logits<Shape32, GRAD, HEAD_SQUARE, true>(a, st);
  return s == HEAD_256 ? logits<Shape256, GRAD>(a, second, st) : logits<Shape128, GRAD>(a, second, st);
}

template <class SX, class SW, bool F32>
hipError_t products(HeadDx x, HeadDw w, hipStream_t st) {
  x.dt = tiles(x.d, SX::BM), x.nt = tiles(x.np, SX::BN);
  w.dt = tiles(w.d, SW::BM), w.vt = tiles(w.cols, SW::BN);
  const int64_t dw_tiles = w.dt * w.vt * w.splits, n = dw_tiles + x.dt * x.nt * x.splits;
  // memory ends first: a tile stands for 128 rows or words of 64 padded columns at least
  if (n * SX::NT >= int64_t(1) << 32) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((head_products_kernel<SX, SW, F32>), dim3(static_cast<unsigned>(n)), dim3(SX::NT), 0, st, x, w, dw_tiles);
  return hipGetLastError();
}

}  // namespace

int64_t head_tile_words(HeadShape s, int64_t vocab) { return s == HEAD_THIN ? thin_run(vocab, 16) : s == HEAD_256 ? Shape256::BM : s == HEAD_128 ? Shape128::BM : Shape32::BM; }
int64_t head_tile_features(HeadShape s) { return s == HEAD_256 ? Shape256::BM : s == HEAD_128 ? Shape128::BM : Shape32::BM; }
int64_t head_tile_rows(HeadShape s) { return s == HEAD_256 ? Shape256::BN : s == HEAD_128 ? Shape128::BN : Shape32::BN; }

hipError_t head_launch_sums(const HeadLogits& a, HeadShape s, HeadSecond second, hipStream_t st) {
  return logits<false>(a, s, second, st);
}
hipError_t head_launch_grad(const HeadLogits& a, HeadShape s, HeadSecond second, hipStream_t st) {
  return logits<true>(a, s, second, st);
}
hipError_t head_launch_products(const HeadDx& x, const HeadDw& w, HeadShape s, hipStream_t st) {
  if (x.f32) return s == HEAD_256 ? products<Shape256, Shape256, true>(x, w, st) : products<Shape128, Shape128, true>(x, w, st);
  return s == HEAD_256   ? products<Shape256, Shape256, false>(x, w, st)
         : s == HEAD_128 ? products<Shape128, Shape128, false>(x, w, st)
                         : products<Shape64, Shape128, false>(x, w, st);
}

int64_t head_few_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }
// two waves a SIMD, of 16 words at least
int64_t head_few_run(int64_t rows, int64_t d, int64_t words) {
  const int64_t cols = tiles(d, rows <= 16 ? 256 : 128), run = tiles(tiles(words * cols, 2048), 4) * 4;
  return run < 16 ? 16 : run;
}
hipError_t head_launch_few(const HeadFew& a, int64_t rows, int64_t run, int64_t splits, hipStream_t st) {
  return rows <= 8 ? few<8, 4>(a, run, splits, st) : rows <= 16 ? few<16, 4>(a, run, splits, st) : few<32, 2>(a, run, splits, st);
}

}  // namespace monarch
