// Pipelined bf16 matrix product (gfx950): the main loop shared by the head loss's
// three products.
//
//   C[m, n] = sum_k A(m, k) B(n, k), tiles of BM x BN, fp32 sums
//
// An operand lies in memory either with k side by side (KC: element (r, k) at
// p + r*ld + k) or with its rows side by side (KM: at p + k*ld + r), so that none of
// x w^T, g w and g^T x needs a transposed copy. K tiles of 64 go from memory straight
// into LDS (global_load_lds_dwordx4: a wave's 64 pieces of 16 bytes land in 1 KB in
// lane order), NST of them, and from there half by half (32 k, one MFMA's) into
// operand registers ahead of their use:
//   tile t: read its second half; multiply its first;
//           wait for tile t+1 and for this wave's reads of tile t; barrier;
//           load tile t+NST into the place of tile t;
//           read the first half of tile t+1; multiply the second half of tile t.
// One barrier a tile, and a wave's matrix instructions never wait for its own LDS reads.
//
// What bounds the 256 x 256 tile is the way from L2 into the CU: measured apart, 4096 x 4096 x
// 131072 takes 1.5 ms a product when every load hits L1. Lines of 128 bytes have to be
// taken whole (K tiles of 32 took 64-byte halves of KC rows, and a KC tile as long as two KM ones).
//
// KC tile: rows of 128 bytes, 16-byte piece q of row r at q ^ ((r / 2) mod 8). A 16-byte read of
// 64 lanes is served in four groups of 16: lanes 0-3, 12-15, 20-23, 24-27, then 4-11, 16-19,
// 28-31, and so on; the 16 rows and pieces of each group fall on all banks. KM tile: rows of
// 2*ROWS bytes, one for each k, read by ds_read_b64_tr_b16 (16 lanes give four rows of 32
// bytes, lane i gets column i of the four); the 32-byte slot of column group t in row k is
// t ^ g(k), g = (k & 3) + 4 ((k >> 3) & 3), so that the 16 rows of such a read fall on all banks.
//
// fp32 operands come as three bf16 planes (a = a0 + a1 + a2, exact: 8 bits of the
// mantissa each) and their product as six products of planes; what is left out is at
// most 2^-23 of |a||b|. Six bf16 products take 6/16 of one fp32 MFMA product's time.
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
  int64_t kvalid = 0;     // valid k of a; KC: zeros are taken beyond, KM: the last valid k's
};

struct PipeProduct {
  PipeOperand a, b;
  const uint16_t* zeros = nullptr;   // 16 bytes of zeros
};

constexpr int kPipeK = 64;   // k of a tile, two halves

__device__ __forceinline__ int pipe_swizzle(int k) { return (k & 3) | (((k >> 3) & 3) << 2); }

// KC: where a row's 16-byte pieces are turned to.
__device__ __forceinline__ int pipe_turn(int r) { return (r >> 1) & 7; }

// The loads and fragment reads of one operand tile of ROWS rows, by NW waves.
template <bool KM, int ROWS, int NW>
struct PipeTile {
  static constexpr int BYTES = ROWS * kPipeK * 2;
  static constexpr int TOTAL = BYTES / 1024;                    // wave loads a stage
  static constexpr int PER = TOTAL >= NW ? TOTAL / NW : 1;      // a wave's own (few: shared, the same bytes twice)
  static_assert(TOTAL <= NW || TOTAL % NW == 0, "whole loads a wave");
  static constexpr int FRAGS = KM ? 2 : 1;                      // LDS reads a fragment
  static constexpr int CHUNKS = ROWS / 8;                       // KM: 16-byte pieces of one k
  static constexpr int MASK = ROWS / 16 < 16 ? ROWS / 16 - 1 : 15;

  const uint16_t* at;         // the tile, the same for the wave's lanes
  uint32_t off[PER];          // this lane's pieces in it, in bytes
  int64_t adv;                // elements from one K tile to the next

  __device__ __forceinline__ static int load_of(int i, int wave) { return TOTAL >= NW ? wave * PER + i : wave % TOTAL; }

  __device__ __forceinline__ void init(const PipeOperand& o, int64_t r0, int64_t k0, int wave, int lane) {
    adv = KM ? kPipeK * o.ld : kPipeK;
    at = KM ? o.p + k0 * o.ld + r0 : o.p + r0 * o.ld + k0;
    // rows beyond the valid ones are taken from a valid place; r0 is valid
    const int64_t room = o.rows - r0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = load_of(i, wave);
      if constexpr (KM) {
        const int k = j * (1024 / (ROWS * 2)) + lane / CHUNKS, pos = lane % CHUNKS;
        const int c = ((((pos >> 1) ^ (pipe_swizzle(k) & MASK)) << 1) | (pos & 1)) * 8;
        off[i] = static_cast<uint32_t>(k * o.ld + (c < room ? c : room - 8)) * 2;
      } else {
        const int r = j * 8 + (lane >> 3);
        const int q = (lane & 7) ^ pipe_turn(r);
        off[i] = static_cast<uint32_t>((r < room ? r : room - 1) * o.ld + q * 8) * 2;
      }
    }
  }

  __device__ __forceinline__ static void load(const void* s, char* to) {
    __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)(s),
                                     (__attribute__((address_space(3))) void*)(to), 16, 0, 0);
  }
  // Loads the tile `by` elements behind this one, whose k are all valid.
  __device__ __forceinline__ void issue(char* to, int wave, int64_t by) const {
    const char* from = reinterpret_cast<const char*>(at + by);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // an address is a scalar base and 32 bits of a lane's own: sums of both are not kept in registers
      uint32_t o = off[i];
      asm volatile("" : "+v"(o));
      load(from + o, to + load_of(i, wave) * 1024);
    }
  }
  // Loads this tile, of which only `valid` > 0 k are.
  __device__ __forceinline__ void issue_cut(const PipeOperand& o, const uint16_t* zeros, char* to, int wave, int lane,
                                            int64_t valid) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const char* s = reinterpret_cast<const char*>(at) + off[i];
      const int j = load_of(i, wave);
      if constexpr (KM) {
        const int64_t over = j * (1024 / (ROWS * 2)) + lane / CHUNKS - (valid - 1);
        if (over > 0) s -= over * o.ld * 2;
      } else {
        if (((lane & 7) ^ pipe_turn(j * 8 + (lane >> 3))) * 8 >= valid) s = reinterpret_cast<const char*>(zeros);
      }
      load(s, to + load_of(i, wave) * 1024);
    }
  }

  // Byte offset in a tile of this lane's reads of fragments t0 + t (t below a power of two that divides t0).
  // KM: the slot bits of an offset are 0 but for the swizzle, so that a fragment's number
  // is one exclusive or away; KC: so is the half of the tile.
  __device__ __forceinline__ static int base(int lane, int t0) {
    const int l15 = lane & 15, lh = lane >> 4;
    if constexpr (KM)
      return ((8 * lh + (l15 >> 2)) * (ROWS * 2) + (l15 & 3) * 8) ^ ((t0 ^ (((l15 >> 2) | (lh << 2)) & MASK)) << 5);
    else
      return t0 * 2048 + l15 * 128 + ((lh ^ pipe_turn(l15)) << 4);
  }
  __device__ __forceinline__ static bf16x8 read(const char* stage, int base, int t, int half) {
    bf16x8 r;
    if constexpr (KM) {
      const char* at = stage + (base ^ (t << 5)) + half * 32 * ROWS * 2;
      typedef __attribute__((address_space(3))) s16x4 Lds;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(at));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(at + 4 * ROWS * 2));
      __builtin_memcpy(&r, &lo, 8);
      __builtin_memcpy(reinterpret_cast<char*>(&r) + 8, &hi, 8);
    } else {
      const u32x4 v = *reinterpret_cast<const u32x4*>(stage + (base ^ (half << 6)) + t * 2048);
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

template <int N, int I = 0, class F>
__device__ __forceinline__ void pipe_each(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    pipe_each<N, I + 1>(f);
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

// Sets a workgroup's sums to 0.
template <class S>
__device__ __forceinline__ void pipe_clear(f32x4 (&acc)[S::FM][S::FN]) {
#pragma unroll
  for (int mi = 0; mi < S::FM; ++mi)
#pragma unroll
    for (int ni = 0; ni < S::FN; ++ni) acc[mi][ni] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// acc[mi][ni], lane l: rows m0 + (wm*FM + mi)*16 + 4*(l/16) + v, column n0 + (wn*FN + ni)*16 + l%16.
// Adds the products of k in [kb, ke) (kb a multiple of 64) to acc. Only a's k may end inside the last
// tile. Ends with a barrier: `lds` is free.
template <class S, bool AKM, bool BKM>
__device__ __forceinline__ void pipe_product_bf16(const PipeProduct& p, int64_t m0, int64_t n0, int64_t kb, int64_t ke,
                                             char* lds, f32x4 (&acc)[S::FM][S::FN]) {
  using TA = PipeTile<AKM, S::BM, S::NW>;
  using TB = PipeTile<BKM, S::BN, S::NW>;
  constexpr int NI = TA::PER + TB::PER, FM = S::FM, FN = S::FN, NST = S::NST;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int ntiles = ke > kb ? static_cast<int>((ke - kb + kPipeK - 1) / kPipeK) : 0;
  if (ntiles == 0) return;
  TA a;
  a.init(p.a, m0, kb, wave, lane);
  TB b;
  b.init(p.b, n0, kb, wave, lane);
  static_assert((FM & (FM - 1)) == 0 && (FN & (FN - 1)) == 0, "fragments of a wave");
  const int ab = TA::base(lane, wm * FM), bb = TB::base(lane, wn * FN);
  // of the last tile's k of a: all, or those before kvalid
  const int64_t last_valid = p.a.kvalid - kb - static_cast<int64_t>(ntiles - 1) * kPipeK;

  auto issue = [&](int st) {
    char* at = lds + st * S::STAGE;
    a.issue(at, wave, 0);
    b.issue(at + TA::BYTES, wave, 0);
    a.at += a.adv, b.at += b.adv;
  };
  auto issue_any = [&](int st, int tile) {
    char* at = lds + st * S::STAGE;
    if (tile == ntiles - 1 && last_valid < kPipeK)
      a.issue_cut(p.a, p.zeros, at, wave, lane, last_valid);
    else
      a.issue(at, wave, 0);
    b.issue(at + TA::BYTES, wave, 0);
    a.at += a.adv, b.at += b.adv;
  };
  bf16x8 fa[2][FM], fb[2][FN];
  auto read = [&](auto half, int st) {
    constexpr int X = decltype(half)::value;
    const char* at = lds + st * S::STAGE;
    // offsets of single fragments are not kept from tile to tile (they would not fit beside the sums)
    int ar = ab, br = bb;
    if constexpr (AKM) asm volatile("" : "+v"(ar));
    if constexpr (BKM) asm volatile("" : "+v"(br));
#pragma unroll
    for (int mi = 0; mi < FM; ++mi) fa[X][mi] = TA::read(at, ar, mi, X);
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) fb[X][ni] = TB::read(at + TA::BYTES, br, ni, X);
  };
  auto multiply = [&](auto half) {
    constexpr int X = decltype(half)::value;
#pragma unroll
    for (int mi = 0; mi < FM; ++mi)
#pragma unroll
      for (int ni = 0; ni < FN; ++ni)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[X][mi], fb[X][ni], acc[mi][ni], 0, 0, 0);
  };
  using First = std::integral_constant<int, 0>;
  using Second = std::integral_constant<int, 1>;
  // Reads and matrix instructions mix freely within a tile (apart, they take twice the time), but the next
  // tile's reads stay behind: mixed in, they cost 4 to 6% (4096 x 4096 x 131072: 15.7 -> 15.3 ms).
  auto multiply_second = [&]() {
    multiply(Second{});
    __builtin_amdgcn_sched_barrier(0);
  };
  auto meet = [&]() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // waits until at most `later` < NST tiles' loads are in flight
  auto landed = [&](int later) {
    asm volatile("" ::: "memory");
    pipe_wait_stages<NI, NST - 1>(later);
    meet();
  };
#pragma unroll 1
  for (int t = 0; t < NST && t < ntiles; ++t) issue_any(t, t);
  landed((ntiles < NST ? ntiles : NST) - 1);
  read(First{}, 0);
  // a tile in the middle: a whole tile is loaded, NST - 2 stay in flight
  auto tile = [&](auto stage) {
    constexpr int ST = decltype(stage)::value;
    read(Second{}, ST);
    multiply(First{});
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(pipe_wait((NST - 2) * NI));
    meet();
    issue(ST);
    read(First{}, ST + 1 == NST ? 0 : ST + 1);
    multiply_second();
  };
  auto last_tile = [&](auto stage, int t) {
    constexpr int ST = decltype(stage)::value;
    if (t >= ntiles) return;
    read(Second{}, ST);
    multiply(First{});
    const int left = ntiles - 2 - t;   // tiles behind t+1
    if (t + 1 < ntiles) {
      landed(left < NST - 2 ? left : NST - 2);
      if (t + NST < ntiles) issue_any(ST, t + NST);
      read(First{}, ST + 1 == NST ? 0 : ST + 1);
    }
    multiply_second();
  };
  int t = 0;
#pragma unroll 1
  for (; t + NST + NST < ntiles; t += NST) pipe_each<NST>([&](auto i) { tile(i); });
#pragma unroll 1
  for (; t < ntiles; t += NST) pipe_each<NST>([&](auto i) { last_tile(i, t + decltype(i)::value); });
  __syncthreads();
}

// The same for fp32 operands in three bf16 planes. A k tile's six products follow each other so that
// each has one operand of the one before:
//   (a2, b0) (a1, b0) (a1, b1) (a0, b1) (a0, b2) (a0, b0)
// and 7 tiles come through LDS for them instead of 12, the operand that stays in registers.
// LDS holds two tiles of either operand. A tile is read into registers by the product
// that takes it up, and the place is given to the operand's tile after next at once:
//   product           0        1      2       3      4      5
//   takes up        a2 b0     a1     b1      a0     b2     b0
//   then loads      a0 b2     a2'    b0      a1'    b0'    b1'     (': of the next k tile)
// No k is cut: the planes are copies that end in zeros.
template <class S, bool AKM, bool BKM>
__device__ __forceinline__ void pipe_product_f32(const PipeProduct& p, int64_t m0, int64_t n0, int64_t kb, int64_t ke,
                                                 char* lds, f32x4 (&acc)[S::FM][S::FN]) {
  using TA = PipeTile<AKM, S::BM, S::NW>;
  using TB = PipeTile<BKM, S::BN, S::NW>;
  constexpr int FM = S::FM, FN = S::FN, LA = TA::PER, LB = TB::PER;
  static_assert(2 * (TA::BYTES + TB::BYTES) <= S::LDS, "two tiles of each operand");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int ktiles = ke > kb ? static_cast<int>((ke - kb + kPipeK - 1) / kPipeK) : 0;
  if (ktiles == 0) return;
  TA a;
  a.init(p.a, m0, kb, wave, lane);
  TB b;
  b.init(p.b, n0, kb, wave, lane);
  const int ab = TA::base(lane, wm * FM), bb = TB::base(lane, wn * FN);
  char* const lds_b = lds + 2 * TA::BYTES;
  bf16x8 fa[2][FM], fb[2][FN];
  auto read_a = [&](auto half, int place) {
    constexpr int X = decltype(half)::value;
    int r = ab;
    asm volatile("" : "+v"(r));
#pragma unroll
    for (int mi = 0; mi < FM; ++mi) fa[X][mi] = TA::read(lds + place * TA::BYTES, r, mi, X);
  };
  auto read_b = [&](auto half, int place) {
    constexpr int X = decltype(half)::value;
    int r = bb;
    asm volatile("" : "+v"(r));
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) fb[X][ni] = TB::read(lds_b + place * TB::BYTES, r, ni, X);
  };
  auto multiply = [&](auto half) {
    constexpr int X = decltype(half)::value;
#pragma unroll
    for (int mi = 0; mi < FM; ++mi)
#pragma unroll
      for (int ni = 0; ni < FN; ++ni)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[X][mi], fb[X][ni], acc[mi][ni], 0, 0, 0);
  };
  using First = std::integral_constant<int, 0>;
  using Second = std::integral_constant<int, 1>;
  auto multiply_second = [&]() {
    multiply(Second{});
    __builtin_amdgcn_sched_barrier(0);
  };
  // places: of a's tiles in the order a2 a1 a0 every second, of b's in the order b0 b1 b2 b0
  int64_t ka = 0, kbo = 0;   // offsets of this k tile in a plane
  int pa = 0;                // place of this k tile's a2 (three tiles a k tile: it alternates)
  auto load_a = [&](int plane, int64_t k, int place) { a.issue(lds + place * TA::BYTES, wave, plane * p.a.plane + k); };
  auto load_b = [&](int plane, int64_t k, int place) { b.issue(lds_b + place * TB::BYTES, wave, plane * p.b.plane + k); };
  // waits until at most the last N loads of this wave are in flight, and for the other waves
  auto landed = [&](auto n) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(pipe_wait(decltype(n)::value));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  using A = std::integral_constant<int, LA>;
  using B = std::integral_constant<int, LB>;
  using AB = std::integral_constant<int, LA + LB>;
  using None = std::integral_constant<int, 0>;
  load_a(2, 0, 0);
  load_b(0, 0, 0);
  load_a(1, 0, 1);
  load_b(1, 0, 1);
  landed(AB{});
  read_a(First{}, 0);
  read_b(First{}, 0);
#pragma unroll 1
  for (int k = 0; k < ktiles; ++k) {
    // behind the last k tile it is loaded again and not read
    const bool more = k + 1 < ktiles;
    const int64_t ka1 = more ? ka + a.adv : ka, kb1 = more ? kbo + b.adv : kbo;
    // 0: a2 b0
    read_a(Second{}, pa);
    read_b(Second{}, 0);
    multiply(First{});
    landed(B{});           // in flight: b1
    load_a(0, ka, pa);
    load_b(2, kbo, 0);
    read_a(First{}, pa ^ 1);
    multiply_second();
    // 1: a1 b0
    read_a(Second{}, pa ^ 1);
    multiply(First{});
    landed(AB{});          // a0, b2
    load_a(2, ka1, pa ^ 1);
    read_b(First{}, 1);
    multiply_second();
    // 2: a1 b1
    read_b(Second{}, 1);
    multiply(First{});
    landed(AB{});          // b2, a2'
    load_b(0, kbo, 1);
    read_a(First{}, pa);
    multiply_second();
    // 3: a0 b1
    read_a(Second{}, pa);
    multiply(First{});
    landed(AB{});          // a2', b0
    load_a(1, ka1, pa);
    read_b(First{}, 0);
    multiply_second();
    // 4: a0 b2
    read_b(Second{}, 0);
    multiply(First{});
    landed(A{});           // a1'
    load_b(0, kb1, 0);
    read_b(First{}, 1);
    multiply_second();
    // 5: a0 b0
    read_b(Second{}, 1);
    multiply(First{});
    landed(None{});
    load_b(1, kb1, 1);
    read_a(First{}, pa ^ 1);
    read_b(First{}, 0);
    multiply_second();
    ka = ka1, kbo = kb1, pa ^= 1;
  }
  landed(None{});   // what was loaded last has to be in LDS before that is used otherwise
}

template <class S, bool AKM, bool BKM, bool F32>
__device__ __forceinline__ void pipe_product(const PipeProduct& p, int64_t m0, int64_t n0, int64_t kb, int64_t ke,
                                             char* lds, f32x4 (&acc)[S::FM][S::FN]) {
  if constexpr (F32)
    pipe_product_f32<S, AKM, BKM>(p, m0, n0, kb, ke, lds, acc);
  else
    pipe_product_bf16<S, AKM, BKM>(p, m0, n0, kb, ke, lds, acc);
}

}  // namespace monarch
