// Row teams: a row of a matrix is held by TEAM threads in 16-byte pieces
// (gfx950). Shared by the row-wise kernels (norms, distillation loss).
#pragma once

#include "common.h"

namespace monarch {

// A 16-byte access whose address is a multiple of the element size only: rows
// of odd widths start anywhere. The compiler lowers it to one 16-byte access
// (global accesses on this target may be unaligned).
typedef u32x4 __attribute__((aligned(2), may_alias)) u32x4_at2;
typedef u32x4 __attribute__((aligned(4), may_alias)) u32x4_at4;

template <typename T> struct PieceOf;
template <> struct PieceOf<float> {
  static constexpr int N = 4;   // elements of 16 bytes
  typedef u32x4_at4 Raw;
  static __device__ __forceinline__ void unpack(const u32x4& r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float (&v)[4]) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]);
    return r;
  }
};
template <> struct PieceOf<uint16_t> {
  static constexpr int N = 8;
  typedef u32x4_at2 Raw;
  static __device__ __forceinline__ void unpack(const u32x4& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&v)[8]) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    return r;
  }
};

// Moves a piece by one element towards its element 0.
template <int N>
__device__ __forceinline__ void drop_first(u32x4& r) {
  if constexpr (N == 4) {
    r = u32x4{r[1], r[2], r[3], 0u};
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) r[i] = (r[i] >> 16) | (r[i + 1] << 16);
    r[3] >>= 16;
  }
}

// How the rows of d elements lie in pieces of N. WHOLE: d is a multiple of N, so
// that pieces are whole and aligned. CUT: rows start and end anywhere, d >= N.
// SHORT: d < N.
enum Rows { WHOLE = 0, CUT = 1, SHORT = 2 };

// Elements [at, at + N) of a row of d elements. A piece past a WHOLE row is 0. A
// piece that a CUT row's end cuts, or that lies past it, is the row's last N
// elements instead, so that every load is one access that nothing waits for: its
// first at + N - d elements belong to the piece before and do not count (mask()
// sets them to 0, store_piece() leaves them out). A SHORT row is loaded an element
// at a time, as its last N elements too.
template <typename T, Rows R>
__device__ __forceinline__ u32x4 load_piece(const T* row, int at, int d) {
  constexpr int N = PieceOf<T>::N;
  if constexpr (R == WHOLE) {
    u32x4 r = {0, 0, 0, 0};
    if (at < d) r = *reinterpret_cast<const u32x4*>(row + static_cast<unsigned>(at));
    return r;
  } else if constexpr (R == CUT) {
    return *reinterpret_cast<const typename PieceOf<T>::Raw*>(row + static_cast<unsigned>(min(at, d - N)));
  } else {
    u32x4 r = {0, 0, 0, 0};
#pragma unroll 1
    for (int i = 0; i < d; ++i) {
      drop_first<N>(r);
      if constexpr (N == 4)
        r[3] = __float_as_uint(row[i]);
      else
        r[3] |= static_cast<uint32_t>(row[i]) << 16;
    }
    return r;
  }
}

// Sets the values of a piece that do not count to 0.
template <Rows R, int N>
__device__ __forceinline__ void mask(float (&v)[N], int at, int d) {
  if constexpr (R == WHOLE) {
    if (at >= d)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.0f;
  } else {
    const int s = at + N - d;
    if (s > 0)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = i < s ? 0.0f : v[i];
  }
}

// Rows are stored past the caches (they are too many to be read back from them,
// and the lines they would take are those of tensors still to be read): 16384 x
// 768 bf16 forward 20.7 -> 18.7 us.
template <typename T, Rows R>
__device__ __forceinline__ void store_piece(T* row, int at, int d, u32x4 r) {
  constexpr int N = PieceOf<T>::N;
  if constexpr (R == WHOLE) {
    if (at < d) __builtin_nontemporal_store(r, reinterpret_cast<u32x4*>(row + static_cast<unsigned>(at)));
    return;
  }
  if (at + N <= d) {
    __builtin_nontemporal_store(r, reinterpret_cast<typename PieceOf<T>::Raw*>(row + static_cast<unsigned>(at)));
    return;
  }
  if (at >= d) return;
#pragma unroll 1
  for (int i = d - N; i < d; ++i) {
    if (i < at) {
      drop_first<N>(r);
      continue;
    }
    if constexpr (N == 4)
      row[i] = __uint_as_float(r[0]);
    else
      row[i] = static_cast<uint16_t>(r[0]);
    drop_first<N>(r);
  }
}

// Keeps the compiler from carrying what it computed from r to the next use of
// r: unpacking again is cheaper than the registers.
__device__ __forceinline__ void forget(u32x4& r) { asm volatile("" : "+v"(r)); }
__device__ __forceinline__ void forget(uint32_t& r) { asm volatile("" : "+v"(r)); }

// A loop-invariant value that is to be computed with anew in every iteration:
// offsets and conditions derived from it would otherwise be kept in registers.
__device__ __forceinline__ int anew(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

template <int CTRL>
__device__ __forceinline__ float dpp_read(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

struct SumOp {
  static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct MaxOp {
  static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

// Reduction over aligned groups of W lanes (16, 32 or 64), the result in every
// lane, in the register file alone: two quad permutations, the half-row and
// row mirrors, then the row and half-wave swaps. The order is fixed.
template <class Op, int W>
__device__ __forceinline__ float lanes_reduce(float v) {
  v = Op::of(v, dpp_read<0xb1>(v));    // quad_perm [1,0,3,2]
  v = Op::of(v, dpp_read<0x4e>(v));    // quad_perm [2,3,0,1]
  v = Op::of(v, dpp_read<0x141>(v));   // row_half_mirror
  v = Op::of(v, dpp_read<0x140>(v));   // row_mirror
  if constexpr (W >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    v = Op::of(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  if constexpr (W >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    v = Op::of(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  return v;
}

// Reductions over a team of TEAM threads (16 .. 1024, a power of two; a team of
// more than a wave is the whole workgroup), in a fixed order. Several values
// go through one exchange. Two LDS slots are used in turn, so one barrier an
// exchange is enough: a wave that writes a slot again has passed the barrier
// of the exchange between, which every reader of the slot reached first.
template <int TEAM>
struct Team {
  static constexpr int WAVES = TEAM > 64 ? TEAM / 64 : 1;
  static constexpr int MAXV = 4;   // values an exchange
  struct Lds {
    float slot[2][MAXV][WAVES];
  };
  Lds* lds;
  int turn = 0;
  __device__ __forceinline__ explicit Team(Lds* l) : lds(l) {}

  template <class Op, int K>
  __device__ __forceinline__ void reduce(float (&v)[K]) {
    static_assert(K <= MAXV, "");
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_reduce<Op, (TEAM < 64 ? TEAM : 64)>(v[k]);
    if constexpr (TEAM > 64) {
      const int wave = threadIdx.x / 64;
      if (threadIdx.x % 64 == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) lds->slot[turn][k][wave] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float s = lds->slot[turn][k][0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s = Op::of(s, lds->slot[turn][k][w]);
        v[k] = s;
      }
      turn ^= 1;
    }
  }
  __device__ __forceinline__ float sum(float x) {
    float v[1] = {x};
    reduce<SumOp, 1>(v);
    return v[0];
  }
};

}  // namespace monarch
