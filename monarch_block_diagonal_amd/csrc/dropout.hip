// Dropout from a counter-based generator, joined to a residual; the mask is never
// stored: the backward pass draws it again.
//
//   y_i = residual_i + (r_i >= t ? x_i * 65536 / (65536 - t) : 0),   t = round(65536 p)
//
// r_i are 16 bits of Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers:
// as easy as 1, 2, 3, 2011) under the seed as key and the counter (i / 8, offset): its
// four words give eight elements, the lower half of word j for element 2j. A call with
// its own offset draws numbers of its own whatever its size. 16 bits an element hold
// p to 2^-16; with whole words of 32 bits the generator's 20 products of 32 bits for
// four elements would take longer than the data (a wave's takes 16 cycles each).
//
// A thread takes a 16-byte piece of each tensor at a time and one draw for it: 8 elements
// in bf16; in fp32 4, of the draw's 8 (the other four are drawn again by the next lane,
// which costs less than 32 bytes a lane did, whose loads each took half of every line).
// Bound by HBM.
#include <math.h>

#include "api_internal.h"
#include "monarch.h"
#include "team.h"

namespace monarch {
namespace {

struct Dropout {
  const void *x, *residual;
  void* y;
  const uint64_t* state;   // (seed, offset) in device memory, or null
  uint64_t seed, offset;
  int64_t n;
  uint32_t threshold;
  float scale;
};

__device__ __forceinline__ void philox_round(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
  const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c[0], b = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
  const uint32_t c1 = c[1], c3 = c[3];
  c[0] = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
  c[1] = static_cast<uint32_t>(b);
  c[2] = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
  c[3] = static_cast<uint32_t>(a);
}

__device__ __forceinline__ void philox(uint64_t at, uint64_t offset, uint64_t seed, uint32_t (&c)[4]) {
  c[0] = static_cast<uint32_t>(at), c[1] = static_cast<uint32_t>(at >> 32);
  c[2] = static_cast<uint32_t>(offset), c[3] = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    philox_round(c, k0, k1);
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
}

// U pieces a thread, 256 pieces apart; `group`: this launch's first workgroup.
template <typename T, bool RES, int U>
__global__ __launch_bounds__(256) void dropout_kernel(Dropout a, int64_t group) {
  constexpr int N = PieceOf<T>::N;
  uint64_t seed = a.seed, offset = a.offset;
  if (a.state) seed = a.state[0], offset = a.state[1];
  const int64_t first = (group + blockIdx.x) * (256 * U) + threadIdx.x;
  const int64_t whole = a.n / N;
  const u32x4* x = static_cast<const u32x4*>(a.x);
  const u32x4* res = static_cast<const u32x4*>(a.residual);
  u32x4* y = static_cast<u32x4*>(a.y);
  u32x4 v[U], r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = first + u * 256;
    if (at < whole) {
      v[u] = __builtin_nontemporal_load(x + at);
      if constexpr (RES) r[u] = __builtin_nontemporal_load(res + at);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = first + u * 256;
    if (at > whole) continue;
    uint32_t c[4];
    philox(static_cast<uint64_t>(at * N) >> 3, offset, seed, c);
    if constexpr (N == 4)
      if (at & 1) c[0] = c[2], c[1] = c[3];
    if (at < whole) {
      float f[N], g[N];
      PieceOf<T>::unpack(v[u], f);
      if constexpr (RES) PieceOf<T>::unpack(r[u], g);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t half = (i & 1) ? c[i >> 1] >> 16 : c[i >> 1] & 0xffffu;
        // chosen, not multiplied: what is dropped may be infinite or NaN
        const float kept = RES ? fmaf(f[i], a.scale, g[i]) : f[i] * a.scale;
        f[i] = half >= a.threshold ? kept : RES ? g[i] : 0.0f;
      }
      __builtin_nontemporal_store(PieceOf<T>::pack(f), y + at);
    } else {
      // the last elements, fewer than a piece
#pragma unroll 1
      for (int64_t i = at * N; i < a.n; ++i) {
        const int e = static_cast<int>(i - at * N);
        const uint32_t word = e < 4 ? (e < 2 ? c[0] : c[1]) : (e < 6 ? c[2] : c[3]);
        const uint32_t half = (e & 1) ? word >> 16 : word & 0xffffu;
        const float g = RES ? Io<T>::load(a.residual, i) : 0.0f;
        const float f = Io<T>::load(a.x, i);
        Io<T>::store(a.y, i, half >= a.threshold ? (RES ? fmaf(f, a.scale, g) : f * a.scale) : g);
      }
    }
  }
}

template <typename T, bool RES>
hipError_t launch(const Dropout& a, hipStream_t s) {
  constexpr int U = 4;
  const int64_t pieces = (a.n + PieceOf<T>::N - 1) / PieceOf<T>::N;
  // few pieces: one a thread, so that every CU has some
  if (pieces <= 256 * 1024) {
    hipLaunchKernelGGL((dropout_kernel<T, RES, 1>), dim3(static_cast<unsigned>((pieces + 255) / 256)), dim3(256), 0, s, a,
                       int64_t(0));
    return hipGetLastError();
  }
  // A launch has fewer than 2^32 threads; 2^21 workgroups are 32 GiB of a tensor.
  constexpr int64_t kMost = int64_t(1) << 21;
  const int64_t groups = (pieces + 256 * U - 1) / (256 * U);
  for (int64_t first = 0; first < groups; first += kMost) {
    const int64_t n = groups - first < kMost ? groups - first : kMost;
    hipLaunchKernelGGL((dropout_kernel<T, RES, U>), dim3(static_cast<unsigned>(n)), dim3(256), 0, s, a, first);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace
}  // namespace monarch

using namespace monarch;

extern "C" int monarch_dropout(const void* x, const void* residual, void* y, int64_t n, double p, uint64_t seed,
                               uint64_t offset, const void* state, int dtype, void* stream, void* const* events,
                               int n_events) {
  if (dtype != MONARCH_F32 && dtype != MONARCH_BF16) return MONARCH_ERR_DTYPE;
  if (n < 0 || n > (int64_t(1) << 41)) return MONARCH_ERR_SHAPE;
  if (!(p >= 0.0) || !(p <= 1.0)) return MONARCH_ERR_VALUE;
  if (n > 0 && (!x || !y)) return MONARCH_ERR_NULL;
  if (misaligned(x) || misaligned(residual) || misaligned(y) || reinterpret_cast<uintptr_t>(state) % 8 != 0)
    return MONARCH_ERR_ALIGN;
  if (n == 0) return MONARCH_OK;
  Dropout a;
  a.x = x, a.residual = residual, a.y = y, a.state = static_cast<const uint64_t*>(state);
  a.seed = seed, a.offset = offset, a.n = n;
  a.threshold = static_cast<uint32_t>(floor(p * 65536.0 + 0.5));
  a.scale = a.threshold < 65536u ? static_cast<float>(65536.0 / (65536.0 - a.threshold)) : 0.0f;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Tracer tr{events, n_events, 0, s};
  int st = record_hip(tr.mark());
  if (st) return st;
  const bool bf16 = dtype == MONARCH_BF16;
  st = record_hip(residual ? (bf16 ? launch<uint16_t, true>(a, s) : launch<float, true>(a, s))
                           : (bf16 ? launch<uint16_t, false>(a, s) : launch<float, false>(a, s)));
  if (st) return st;
  return record_hip(tr.mark());
}
