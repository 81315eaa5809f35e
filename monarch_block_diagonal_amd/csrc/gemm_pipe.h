// Pipelined bf16 matrix product (gfx950): the main loop shared by the head loss's
// three products.
//
//   C[m, n] = sum_k A(m, k) B(n, k), tiles of BM x BN, fp32 sums
//
// An operand lies in memory either with k side by side (KC: element (r, k) at
// p + r*ld + k) or with its rows side by side (KM: at p + k*ld + r), so that none of
// x w^T, g w and g^T x needs a transposed copy. K tiles of 32 go from memory straight
// into LDS (global_load_lds_dwordx4: a wave's 64 pieces of 16 bytes land in 1 KB in
// lane order), NST stages deep, and from there into MFMA operands a step ahead of
// their use, so that a wave's matrix instructions never wait for its own LDS reads:
//   step s: wait for the loads of stage s+1 and this wave's reads of stage s; barrier;
//           load stage s+NST into the place of stage s; read stage s+1 into registers;
//           multiply stage s.
// One barrier a step, no wait for the loads of later stages.
//
// KC stage: rows of 64 bytes, 16-byte piece q of row r at q ^ ((r >> 2) & 3): the 16
// rows of a fragment read fall on all banks. KM stage: rows of 2*ROWS bytes, one for
// each k, read by ds_read_b64_tr_b16 (16 lanes give four rows of 32 bytes, lane i gets
// column i of the four); the 32-byte slot of column group t in row k is t ^ g(k), g =
// (k & 3) + 4 ((k >> 3) & 3), so that the 16 rows of such a read fall on all banks.
//
// fp32 operands come as three bf16 planes (a = a0 + a1 + a2, exact: 8 bits of the
// mantissa each) and their product as six products of planes, least first; what is
// left out is at most 2^-23 of |a||b|. Six bf16 products take 6/16 of one fp32 MFMA product's time.
#pragma once

#include <type_traits>

#include "common.h"

namespace monarch {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// One operand as it lies in memory (elements of bf16).
struct PipeOperand {
  const uint16_t* p = nullptr;
  int64_t ld = 0;
  int64_t plane = 0;      // from one bf16 plane to the next (fp32)
  int64_t rows = 0;       // valid rows (m or n); others are read from a valid place
  int64_t kvalid = 0;     // valid k; KC: zeros are taken beyond, KM: the last valid k's
};

struct PipeProduct {
  PipeOperand a, b;
  const uint16_t* zeros = nullptr;   // 16 bytes of zeros
  int planes = 1;                    // 1: bf16, 3: fp32 as three planes
};

constexpr int kPipeK = 32;

__device__ __forceinline__ int pipe_swizzle(int k) { return (k & 3) | (((k >> 3) & 3) << 2); }

// The loads and fragment reads of one operand tile of ROWS rows, by NW waves.
template <bool KM, int ROWS, int NW>
struct PipeTile {
  static constexpr int BYTES = ROWS * kPipeK * 2;
  static constexpr int TOTAL = BYTES / 1024;                    // wave loads a stage
  static constexpr int PER = TOTAL >= NW ? TOTAL / NW : 1;      // a wave's own (few: shared, the same bytes twice)
  static_assert(TOTAL <= NW || TOTAL % NW == 0, "whole loads a wave");
  static constexpr int CHUNKS = ROWS / 8;                       // KM: 16-byte pieces of one k
  static constexpr int MASK = ROWS / 16 < 16 ? ROWS / 16 - 1 : 15;

  const uint16_t* ptr[PER];
  int kq[PER];   // this lane's k within a tile (KC: of its piece's first element)
  int lds[PER];  // byte offset of the wave's load
  int64_t ld;

  __device__ __forceinline__ void init(const PipeOperand& o, int64_t r0, int wave, int lane) {
    ld = o.ld;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = TOTAL >= NW ? wave * PER + i : wave % TOTAL;
      lds[i] = j * 1024;
      if constexpr (KM) {
        const int k = j * (1024 / (ROWS * 2)) + lane / CHUNKS, pos = lane % CHUNKS;
        const int c = ((((pos >> 1) ^ (pipe_swizzle(k) & MASK)) << 1) | (pos & 1)) * 8;
        kq[i] = k;
        ptr[i] = o.p + k * ld + (r0 + c < o.rows ? r0 + c : 0);
      } else {
        const int r = j * 16 + (lane >> 2);
        const int q = (lane & 3) ^ ((r >> 2) & 3);
        kq[i] = q * 8;
        const int64_t row = r0 + r < o.rows ? r0 + r : o.rows - 1;
        ptr[i] = o.p + row * ld + q * 8;
      }
    }
  }

  // Loads the tile at k0 (`off`: its plane's offset).
  __device__ __forceinline__ void issue(const PipeOperand& o, const uint16_t* zeros, char* stage, int64_t k0,
                                        int64_t off) {
    const bool tail = k0 + kPipeK > o.kvalid;
    const int64_t step = off + (KM ? k0 * ld : k0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint16_t* s = ptr[i] + step;
      if (tail) {
        if constexpr (KM) {
          const int64_t over = k0 + kq[i] - (o.kvalid - 1);
          if (over > 0) s -= over * ld;
        } else {
          if (k0 + kq[i] >= o.kvalid) s = zeros;
        }
      }
      __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)(s),
                                       (__attribute__((address_space(3))) void*)(stage + lds[i]), 16, 0, 0);
    }
  }

  // Byte offset of this lane's fragment reads (tile t of 16 rows adds frag()).
  __device__ __forceinline__ static int base(int lane) {
    const int l15 = lane & 15, lh = lane >> 4;
    if constexpr (KM)
      return (8 * lh + (l15 >> 2)) * (ROWS * 2) + (l15 & 3) * 8;
    else
      return l15 * 64 + ((lh ^ ((l15 >> 2) & 3)) << 4);
  }
  __device__ __forceinline__ static bf16x8 read(const char* stage, int base, int t, int lane) {
    bf16x8 r;
    if constexpr (KM) {
      const int g = (((lane & 15) >> 2) | ((lane >> 4) << 2)) & MASK;
      const char* at = stage + base + ((t ^ g) << 5);
      typedef __attribute__((address_space(3))) s16x4 Lds;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(at));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(at + 4 * ROWS * 2));
      __builtin_memcpy(&r, &lo, 8);
      __builtin_memcpy(reinterpret_cast<char*>(&r) + 8, &hi, 8);
    } else {
      const u32x4 v = *reinterpret_cast<const u32x4*>(stage + base + t * 1024);
      __builtin_memcpy(&r, &v, 16);
    }
    return r;
  }
};

// s_waitcnt: vector memory count <= n, LDS count 0, export count untouched
constexpr int pipe_wait(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4); }

template <int NI, int MOST>
__device__ __forceinline__ void pipe_wait_stages(int later) {
  static_assert(NI * MOST < 64, "vmcnt has six bits");
  if constexpr (MOST > 0) {
    if (later >= MOST)
      __builtin_amdgcn_s_waitcnt(pipe_wait(MOST * NI));
    else
      pipe_wait_stages<NI, MOST - 1>(later);
  } else {
    __builtin_amdgcn_s_waitcnt(pipe_wait(0));
  }
}

// WM x WN waves of FM x FN tiles of 16 x 16.
template <int WM_, int WN_, int FM_, int FN_, int NST_>
struct PipeShape {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_, NST = NST_;
  static constexpr int BM = WM * FM * 16, BN = WN * FN * 16, NW = WM * WN, NT = NW * 64;
  static constexpr int STAGE = (BM + BN) * kPipeK * 2;
  static constexpr int LDS = STAGE * NST;
};

// acc[mi][ni], lane l: rows m0 + (wm*FM + mi)*16 + 4*(l/16) + v, column n0 + (wn*FN + ni)*16 + l%16.
// Sums k in [kb, ke) (kb a multiple of 32). Ends with a barrier: `lds` is free.
template <class S, bool AKM, bool BKM>
__device__ __forceinline__ void pipe_product(const PipeProduct& p, int64_t m0, int64_t n0, int64_t kb, int64_t ke,
                                             char* lds, f32x4 (&acc)[S::FM][S::FN]) {
  using TA = PipeTile<AKM, S::BM, S::NW>;
  using TB = PipeTile<BKM, S::BN, S::NW>;
  constexpr int NI = TA::PER + TB::PER, FM = S::FM, FN = S::FN, NST = S::NST;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
#pragma unroll
  for (int mi = 0; mi < FM; ++mi)
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int ksteps = ke > kb ? static_cast<int>((ke - kb + kPipeK - 1) / kPipeK) : 0;
  const int nsteps = ksteps * (p.planes == 1 ? 1 : 6);
  if (nsteps == 0) return;
  TA a;
  a.init(p.a, m0, wave, lane);
  TB b;
  b.init(p.b, n0, wave, lane);
  const int ab = TA::base(lane), bb = TB::base(lane);

  // planes of A and B in the order of their products: (2,0) (0,2) (1,1) (1,0) (0,1) (0,0)
  int ik = 0, iseg = 0;   // the next tile to load
  uint32_t seqa = 0x001102, seqb = 0x010120;
  int64_t offa = p.planes == 1 ? 0 : 2 * p.a.plane, offb = 0;
  auto issue = [&](int st) {
    char* at = lds + st * S::STAGE;
    const int64_t k0 = kb + static_cast<int64_t>(ik) * kPipeK;
    a.issue(p.a, p.zeros, at, k0, offa);
    b.issue(p.b, p.zeros, at + TA::BYTES, k0, offb);
    if (++ik == ksteps) {
      ik = 0, ++iseg;
      if (p.planes != 1) {
        offa = ((seqa >> (4 * iseg)) & 3) * p.a.plane;
        offb = ((seqb >> (4 * iseg)) & 3) * p.b.plane;
      }
    }
  };
  bf16x8 fa[2][FM], fb[2][FN];
  auto read = [&](auto slot, int st) {
    constexpr int X = decltype(slot)::value;
    const char* at = lds + st * S::STAGE;
#pragma unroll
    for (int mi = 0; mi < FM; ++mi) fa[X][mi] = TA::read(at, ab, wm * FM + mi, lane);
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) fb[X][ni] = TB::read(at + TA::BYTES, bb, wn * FN + ni, lane);
  };
  auto multiply = [&](auto slot) {
    constexpr int X = decltype(slot)::value;
#pragma unroll
    for (int mi = 0; mi < FM; ++mi)
#pragma unroll
      for (int ni = 0; ni < FN; ++ni)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[X][mi], fb[X][ni], acc[mi][ni], 0, 0, 0);
  };
  // waits until at most `later` < NST stages' loads are in flight
  auto landed = [&](int later) {
    asm volatile("" ::: "memory");
    pipe_wait_stages<NI, NST - 1>(later);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  using Zero = std::integral_constant<int, 0>;
  using One = std::integral_constant<int, 1>;
  constexpr int AHEAD = NST;   // stages loaded before the first step
#pragma unroll 1
  for (int s = 0; s < AHEAD && s < nsteps; ++s) issue(s);
  landed((nsteps < AHEAD ? nsteps : AHEAD) - 1);
  read(Zero{}, 0);
  int st = 0;   // stage of step s
  auto step = [&](auto now, auto next, int s) {
    const int left = nsteps - 2 - s;   // stages behind s+1
    const int st1 = st + 1 == NST ? 0 : st + 1;
    if (s + 1 < nsteps) {
      landed(left < NST - 2 ? left : NST - 2);
      if (s + NST < nsteps) issue(st);
      read(next, st1);
    }
    multiply(now);
    st = st1;
  };
#pragma unroll 1
  for (int s = 0; s < nsteps; s += 2) {
    step(Zero{}, One{}, s);
    if (s + 1 < nsteps) step(One{}, Zero{}, s + 1);
  }
  __syncthreads();
}

}  // namespace monarch
