// Distillation from a teacher's top logits: loss and gradient.
//
// For a row of student logits z [V], teacher entries (id_k, t_k), a label c, a
// temperature T and a mix:
//   p_k = softmax over the valid entries of t_k / T
//   q = softmax(z / T), s = softmax(z)
//   loss = mix T^2 sum_k p_k (log p_k - log q[id_k]) - (1 - mix) log s[c]
//   dz_j = w (mix T (q_j - sum_{k: id_k = j} p_k) + (1 - mix) (s_j - [j = c]))
// An entry is valid with 0 <= id < V and t > -inf, a label with 0 <= c < V; without a
// valid entry the first term is absent, without a label the second. A row with
// neither, or whose logits are -inf throughout, has loss 0 and gradient 0.
//
// A workgroup takes a row. The row is cut at its 16-byte boundaries into whole
// pieces, of which every thread holds up to P in registers from its sums to its
// gradient (a row that is longer streams the rest twice), and at most 7 elements
// before and 7 behind them, one for each of the first threads. Exponentials are
// 2^((z - m) log2(e) / T) with m the row's maximum: z - m is exact or rounded once,
// and rows of the type's lowest value (m huge) stay finite. Sums are fp32.
//
// Loss and gradient together read and write each logit once: bound by HBM while
// every CU has many rows to take, by the phases of a row (load, about 20 operations a
// logit, store) where it has few. Measured (a call among others): loss of 4096 x 50257
// bf16 at T = 2 with labels 77 us, 5.4 TB/s (its arithmetic busy 86% of the time, but no
// slower than T = 1, which has a tenth less); both of 16384 x 50257 bf16 588 us, 5.6
// TB/s, which a copy of that size reaches (40 calls timed one by one: median 595, 583 to
// 625; in kernel traces, which run them apart, medians 621 to 642, 593 at least); of 1024 x 50257 bf16 (4
// rows a CU) 48 us, 4.3 TB/s; of 1000 x 10000 fp32 26.6 us; of 2048 x 131072 fp32, which no
// CU holds, 486 us, 4.4 TB/s. Read twice instead of held, the second took 784 us and the
// last 718.
// Kept out by measurement: workgroups that load their next row into the registers
// that a gradient frees (621 -> 672 us: the waits at a row's start then cover its
// stores), and 2^(z c - M) as one fused operation with a second path for rows far
// from 0 (no gain).
#include <math.h>

#include "api_internal.h"
#include "monarch.h"
#include "team.h"

namespace monarch {
namespace {

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr float kLog2e = 1.44269504088896340736f;

struct Distill {
  const void* z;
  const float* teacher;
  const int64_t* ids;
  const int64_t* labels;    // null: none
  const float* weight;      // null: 1 (the step) -- dloss of the backward pass
  const float* stats_in;    // backward: (m, sum at T, sum at 1, unused) a row
  float *loss, *stats;      // forward
  void* dz;
  int64_t rows, ld, dld;
  int vocab, top;
  float temperature, mix;
};

// LDS slots for the entries and the label, in whole 16-byte reads.
__host__ __device__ inline int entry_slots(int top) { return (top + 4) / 4 * 4; }

enum { WITH_LOSS = 1, WITH_GRAD = 2 };   // loss and sums from z; gradient

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The second softmax of a row, that of the labels' term, beside the one at T.
enum Second {
  NONE = 0,     // no label term, or T = 1: one softmax
  OWN = 1,      // its own exponentials
  SQUARE = 2    // T = 2, the usual one: e^z = (e^(z/2))^2, a product and no second
                // exponential (4096 x 50257 bf16, loss: 88 us with OWN, 77 us; both: 184, 171)
};

// Maximum and sums of exponentials of one thread's share of a row. The maximum
// rises a piece at a time: one more exponential for every piece, and the sums
// of the first pieces are under way while the last ones are loaded.
template <int SECOND>
struct Running {
  float m = -3.402823466e38f, st = 0.0f, s1 = 0.0f;
  __device__ __forceinline__ void raise(float to, float ct) {
    const float f = exp2_of((m - to) * ct);
    st *= f;
    if constexpr (SECOND == OWN) s1 *= exp2_of((m - to) * kLog2e);
    if constexpr (SECOND == SQUARE) s1 *= f * f;
    m = to;
  }
  __device__ __forceinline__ void add(float v, float ct) {
    const float e = exp2_of((v - m) * ct);
    st += e;
    if constexpr (SECOND == OWN) s1 += exp2_of((v - m) * kLog2e);
    if constexpr (SECOND == SQUARE) s1 = fmaf(e, e, s1);
  }
  template <int N>
  __device__ __forceinline__ void add_piece(const float (&v)[N], float ct) {
    float to = m;
#pragma unroll
    for (int i = 0; i < N; i += 2) to = fmaxf(fmaxf(to, v[i]), v[i + 1]);
    raise(to, ct);
#pragma unroll
    for (int i = 0; i < N; ++i) add(v[i], ct);
  }
};

template <typename T, int TEAM, int P, int WHAT, int SECOND>
__global__ __launch_bounds__(TEAM, 4) void distill_kernel(Distill a) {
  constexpr int N = PieceOf<T>::N, U = 4;
  // rows longer than 1024 threads' registers: the next 8 rounds stay in LDS (128 KB)
  constexpr int L = TEAM == 1024 && WHAT == (WITH_LOSS | WITH_GRAD) ? 8 : 0;
  static_assert(L % U == 0, "");
  __shared__ u32x4 s_held[L > 0 ? L * TEAM : 1];
  constexpr int PR = P > 0 ? P : 1;
  constexpr uint32_t kMinusInf = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  const u32x4 nothing_more = {kMinusInf, kMinusInf, kMinusInf, kMinusInf};   // adds nothing
  // `top` entries and the label: column (-1: none), student's logit, teacher's
  // exponential; then the teacher's logits
  extern __shared__ __align__(16) int s_id[];
  __shared__ typename Team<TEAM>::Lds tlds;
  const int slots = entry_slots(a.top);
  float* s_z = reinterpret_cast<float*>(s_id + slots);
  float* s_e = s_z + slots;
  float* s_t = s_e + slots;
  Team<TEAM> team(&tlds);
  const unsigned lane = threadIdx.x;   // unsigned: an offset from a scalar address
  const int tid = static_cast<int>(lane);
  const float ct = kLog2e / a.temperature;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    // the row's whole pieces start `head` elements in; `extra` is this thread's
    // element before or behind them
    int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / int(sizeof(T));
    if (head > a.vocab) head = a.vocab;
    const int pieces = (a.vocab - head) / N;
    const int extra = tid < head ? tid : tid + pieces * N;
    const bool has_extra = tid < 2 * N && extra < a.vocab;
    const u32x4* body = reinterpret_cast<const u32x4*>(z + head);

    // this thread's entry, the label and the single elements first: loads return
    // in order, and these few are wanted as soon as the pieces are here
    int64_t id0 = -1;
    float t0 = 0.0f;
    if (tid < a.top) {
      id0 = a.ids[row * a.top + tid];
      t0 = a.teacher[row * a.top + tid];
    }
    const int64_t label = a.labels ? a.labels[row] : -1;
    const bool told = label >= 0 && label < a.vocab && a.mix < 1.0f;
    const float ze = has_extra ? Io<T>::load(z, extra) : -INFINITY;
    // P rounds of TEAM pieces, loaded without a branch between them: the last,
    // short round is moved back to end with the row (its first threads then hold
    // pieces of the round before, which do not count), and those past it repeat it
    u32x4 raw[PR];
    if (P > 0 && pieces >= TEAM) {
#pragma unroll
      for (int p = 0; p < P; ++p) raw[p] = (body + min(p * TEAM, pieces - TEAM))[lane];
    } else if (P > 0 && tid < pieces) {
      raw[0] = body[lane];
    }
    // where round p starts, and whether this thread's piece in it counts
    auto round_at = [](int p, int np) { return min(p * TEAM, max(np - TEAM, 0)); };
    auto counts = [tid](int p, int at, int np) { return at + tid >= p * TEAM && at + tid < np; };

    float m, st, s1;
    Running<SECOND> r;
    // the number of pieces is read anew for every pass over them: one kernel
    // body for each number of them costs registers
    int np = anew(pieces);
    if constexpr (WHAT & WITH_LOSS) {
      r.raise(fmaxf(r.m, ze), ct);
      r.add(ze, ct);
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (p * TEAM < np) {
          if (p * TEAM + TEAM > np && !counts(p, round_at(p, np), np)) raw[p] = nothing_more;
          float v[N];
          PieceOf<T>::unpack(raw[p], v);
          r.template add_piece<N>(v, ct);
          if (WHAT & WITH_GRAD) forget(raw[p]);
        }
      for (int base = P * TEAM; base < pieces; base += TEAM * U) {
        u32x4 more[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          more[u] = nothing_more;
          if (base + u * TEAM + tid < pieces) more[u] = (body + (base + u * TEAM))[lane];
        }
        if (base < (P + L) * TEAM)
#pragma unroll
          for (int u = 0; u < U; ++u) s_held[base - P * TEAM + u * TEAM + tid] = more[u];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (base + u * TEAM < pieces) {
            float v[N];
            PieceOf<T>::unpack(more[u], v);
            r.template add_piece<N>(v, ct);
          }
      }
    }
    // the teacher's entries and the student's logits there
    float tmax = -INFINITY;
    for (int k = tid; k < slots; k += TEAM) {
      int id = -1;
      float t = 0.0f;
      if (k < a.top) {
        const int64_t id64 = k == tid ? id0 : a.ids[row * a.top + k];
        t = k == tid ? t0 : a.teacher[row * a.top + k];
        if (id64 >= 0 && id64 < a.vocab && t > -INFINITY) {
          id = static_cast<int>(id64);
          tmax = fmaxf(tmax, t);
        }
      } else if (k == a.top && told) {
        id = static_cast<int>(label);
      }
      s_id[k] = id;
      s_t[k] = t;
      s_z[k] = id >= 0 ? Io<T>::load(z, id) : 0.0f;
    }
    if constexpr (WHAT & WITH_LOSS) {
      float top2[2] = {r.m, tmax};
      team.template reduce<MaxOp, 2>(top2);
      m = top2[0];
      tmax = top2[1];
      r.raise(m, ct);
    } else {
      float top1[1] = {tmax};
      team.template reduce<MaxOp, 1>(top1);
      tmax = top1[0];
      const f32x4 sums = *reinterpret_cast<const f32x4*>(a.stats_in + row * 4);
      m = sums[0];
      r.st = sums[1];
      r.s1 = sums[2];
    }
    // the teacher's sum, and 2^-10 sum_k e_k ((t_k - tmax) - (z_k - m)): T times the part
    // of sum_k p_k (log p_k - log q_k) that is not T (log st - log tsum). Neither the sum
    // of up to 512 entries nor a quotient by a small T overflows where they name
    // logits of the type's lowest value.
    const bool some = tmax > -INFINITY && a.mix > 0.0f;
    float sums[4] = {0.0f, 0.0f, r.st, r.s1};
    for (int k = tid; k < slots; k += TEAM) {
      float e = 0.0f;
      if (k < a.top && s_id[k] >= 0) {
        const float t = s_t[k] - tmax;
        e = exp2_of(t * ct);
        sums[0] += e;
        if (!(e == 0.0f)) sums[1] = fmaf(e * 0x1p-10f, t - (s_z[k] - m), sums[1]);
      }
      s_e[k] = e;
    }
    if (TEAM <= 64) __syncthreads();   // the entries, which larger teams pass a barrier after
    if constexpr (WHAT & WITH_LOSS) {
      team.template reduce<SumOp, 4>(sums);
      st = sums[2];
      s1 = SECOND == NONE ? st : sums[3];
    } else {
      float tsum[1] = {sums[0]};
      team.template reduce<SumOp, 1>(tsum);
      sums[0] = tsum[0];
      st = r.st;
      s1 = r.s1;
    }
    const bool alive = st != 0.0f;   // NaN counts as alive: it has to come out
    if constexpr (WHAT & WITH_LOSS) {
      if (tid == 0) {
        float loss = 0.0f;
        if (some && alive)
          loss = a.mix * a.temperature * 0x1p10f * (sums[1] / sums[0]) +
                 a.mix * a.temperature * a.temperature * (logf(st) - logf(sums[0]));
        if (told && alive) loss += (1.0f - a.mix) * (logf(s1) - (s_z[a.top] - m));
        a.loss[row] = loss;
        if (a.stats) *reinterpret_cast<f32x4*>(a.stats + row * 4) = f32x4{m, st, s1, 0.0f};
      }
    }
    if constexpr (WHAT & WITH_GRAD) {
      const float w = a.weight ? a.weight[row] : 1.0f;
      const float ga = some && alive ? w * a.mix * a.temperature : 0.0f;
      const float gb = told && alive ? w * (1.0f - a.mix) : 0.0f;
      // one softmax for both terms where they share it
      const float fa = SECOND == NONE ? (ga + gb) / st : ga / st;
      const float fb = SECOND == NONE ? 0.0f : gb / s1;
      T* dz = static_cast<T*>(a.dz) + row * a.dld;
      T* dbody = dz + head;
      const bool nothing = (!some && !told) || !alive;
      auto grad = [&](float v) {
        const float e = exp2_of((v - m) * ct);
        if constexpr (SECOND == OWN) return fmaf(fb, exp2_of((v - m) * kLog2e), fa * e);
        if constexpr (SECOND == SQUARE) return e * fmaf(fb, e, fa);
        return fa * e;
      };
      np = anew(pieces);
      auto put = [&](int first, bool mine, const u32x4& piece) {
        float v[N];
        PieceOf<T>::unpack(piece, v);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = grad(v[i]);
        u32x4 o = PieceOf<T>::pack(v);
        if (nothing) o = u32x4{0, 0, 0, 0};
        if (mine)
          __builtin_nontemporal_store(
              o, reinterpret_cast<typename PieceOf<T>::Raw*>(dbody + static_cast<int64_t>(first) * N) + lane);
      };
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (p * TEAM < np) put(round_at(p, np), counts(p, round_at(p, np), np), raw[p]);
      for (int base = P * TEAM; base < pieces; base += TEAM * U) {
        u32x4 more[U] = {};
        if (base < (P + L) * TEAM) {
#pragma unroll
          for (int u = 0; u < U; ++u) more[u] = s_held[base - P * TEAM + u * TEAM + tid];
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (base + u * TEAM + tid < pieces) more[u] = (body + (base + u * TEAM))[lane];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (base + u * TEAM < pieces)
            put(base + u * TEAM, base + u * TEAM + tid < pieces, more[u]);
      }
      if (has_extra) Io<T>::store(dz, extra, nothing ? 0.0f : grad(ze));
      // the entries and the label: their elements are written again, whole, by the
      // first slot that names them, with the sum of all that do
      const float inv_t = some ? 1.0f / sums[0] : 0.0f;
      auto fix = [&](int k, float& g) {
        const int id = nothing ? -1 : s_id[k];
        float e = s_e[k];
        int same = 0, before = 0;
        for (int j = 0; j < slots; j += 4) {
          const int4 other = *reinterpret_cast<const int4*>(s_id + j);
          same += (other.x == id) + (other.y == id) + (other.z == id) + (other.w == id);
          before += (other.x == id && j < k) + (other.y == id && j + 1 < k) +
                    (other.z == id && j + 2 < k) + (other.w == id && j + 3 < k);
        }
        if (id < 0 || before) return -1;
        if (same > 1) {
          e = 0.0f;
          for (int j = 0; j < slots; ++j)
            if (s_id[j] == id) e += s_e[j];
        }
        g = grad(s_z[k]) - ga * (e * inv_t);
        if (told && id == label) g -= gb;
        return id;
      };
      float g = 0.0f;
      int id = tid < slots ? fix(tid, g) : -1;
      __syncthreads();   // the row is written
      if (id >= 0) Io<T>::store(dz, id, g);
      for (int k = tid + TEAM; k < slots; k += TEAM) {
        id = fix(k, g);
        if (id >= 0) Io<T>::store(dz, id, g);
      }
    }
    __syncthreads();   // the next row overwrites the entries
  }
}

int check_sizes(int64_t rows, int64_t vocab, int64_t ld, int64_t top, int dtype) {
  if (dtype != MONARCH_F32 && dtype != MONARCH_BF16) return MONARCH_ERR_DTYPE;
  // columns are counted in 32 bits, up to a workgroup past the row
  if (rows < 0 || rows >= kLimit || vocab <= 0 || vocab > kLimit / 2 || ld < vocab || top < 0 ||
      top > MONARCH_DISTILL_MAX_TOP)
    return MONARCH_ERR_SHAPE;
  return MONARCH_OK;
}

bool off_elements(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) != 0;
}

template <typename T, int TEAM, int P, int WHAT>
hipError_t launch_second(const Distill& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : (1 << 20))), block(TEAM);
  const size_t lds = static_cast<size_t>(entry_slots(a.top)) * 16;
  const bool two = a.labels && a.mix < 1.0f && a.temperature != 1.0f;
  if (two && a.temperature == 2.0f)
    hipLaunchKernelGGL((distill_kernel<T, TEAM, P, WHAT, SQUARE>), grid, block, lds, s, a);
  else if (two)
    hipLaunchKernelGGL((distill_kernel<T, TEAM, P, WHAT, OWN>), grid, block, lds, s, a);
  else
    hipLaunchKernelGGL((distill_kernel<T, TEAM, P, WHAT, NONE>), grid, block, lds, s, a);
  return hipGetLastError();
}

// The smallest workgroup whose registers hold the row, 4 or 16 pieces a thread
// (1000 x 10000 fp32 step: 256 threads x 16 24 us, 512 x 8 32 us, 1024 x 4 58 us). A
// gradient alone streams the row once, and needs no more than enough threads.
template <typename T, int WHAT>
hipError_t launch_sized(const Distill& a, hipStream_t s) {
  const int pieces = a.vocab / PieceOf<T>::N;
  constexpr bool HOLD = WHAT & WITH_LOSS;
  if (pieces <= 64 * 4) return launch_second<T, 64, HOLD ? 4 : 0, WHAT>(a, s);
  if (pieces <= 256 * 4) return launch_second<T, 256, HOLD ? 4 : 0, WHAT>(a, s);
  if constexpr (HOLD) {
    if (pieces <= 256 * 16) return launch_second<T, 256, 16, WHAT>(a, s);
    if (pieces <= 512 * 16) return launch_second<T, 512, 16, WHAT>(a, s);
    return launch_second<T, 1024, 16, WHAT>(a, s);
  } else {
    return launch_second<T, 512, 0, WHAT>(a, s);
  }
}

template <int WHAT>
hipError_t launch(const Distill& a, bool bf16, hipStream_t s) {
  return bf16 ? launch_sized<uint16_t, WHAT>(a, s) : launch_sized<float, WHAT>(a, s);
}

// The checks that every call shares; `what` as for the kernel.
int check_call(const Distill& a, const void* ids, int what, int dtype, float temperature, float mix) {
  int st = check_sizes(a.rows, a.vocab, a.ld, a.top, dtype);
  if (st) return st;
  if ((what & WITH_GRAD) && a.dld < a.vocab) return MONARCH_ERR_SHAPE;
  if (!(temperature >= 1e-6f) || !(temperature <= 1e6f) || !(mix >= 0.0f) || !(mix <= 1.0f))
    return MONARCH_ERR_VALUE;
  if (a.rows > 0) {
    if (!a.z || (a.top > 0 && (!a.teacher || !ids))) return MONARCH_ERR_NULL;
    if ((what & WITH_LOSS) && !a.loss) return MONARCH_ERR_NULL;
    if ((what & WITH_GRAD) && !a.dz) return MONARCH_ERR_NULL;
    if (what == WITH_GRAD && (!a.stats_in || !a.weight)) return MONARCH_ERR_NULL;
  }
  const int es = dtype == MONARCH_BF16 ? 2 : 4;
  if (off_elements(a.z, es) || off_elements(a.dz, es) || off_elements(a.teacher, 4) ||
      off_elements(ids, 8) || off_elements(a.labels, 8) || off_elements(a.weight, 4) ||
      off_elements(a.loss, 4) || misaligned(a.stats) || misaligned(a.stats_in))
    return MONARCH_ERR_ALIGN;
  return MONARCH_OK;
}

template <int WHAT>
int run_call(Distill a, const void* ids, const void* labels, int64_t vocab, int64_t top,
             float temperature, float mix, int dtype, void* stream, void* const* events,
             int n_events) {
  // sizes first: `vocab` and `top` are kept in 32 bits
  int st = check_sizes(a.rows, vocab, a.ld, top, dtype);
  if (st) return st;
  a.vocab = static_cast<int>(vocab);
  a.top = static_cast<int>(top);
  a.temperature = temperature;
  a.mix = mix;
  a.ids = static_cast<const int64_t*>(ids);
  a.labels = static_cast<const int64_t*>(labels);
  st = check_call(a, ids, WHAT, dtype, temperature, mix);
  if (st) return st;
  if (a.rows == 0) return MONARCH_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Tracer tr{events, n_events, 0, s};
  st = record_hip(tr.mark());
  if (st) return st;
  st = record_hip(launch<WHAT>(a, dtype == MONARCH_BF16, s));
  if (st) return st;
  return record_hip(tr.mark());
}

}  // namespace
}  // namespace monarch

using namespace monarch;

extern "C" {

int monarch_distill_fwd(const void* logits, int64_t ld, const void* teacher, const void* ids,
                        const void* labels, void* loss, void* stats, int64_t rows, int64_t vocab,
                        int64_t top, float temperature, float mix, int dtype, void* stream,
                        void* const* events, int n_events) {
  Distill a = {};
  a.z = logits, a.ld = ld, a.rows = rows;
  a.teacher = static_cast<const float*>(teacher);
  a.loss = static_cast<float*>(loss), a.stats = static_cast<float*>(stats);
  return run_call<WITH_LOSS>(a, ids, labels, vocab, top, temperature, mix, dtype, stream, events,
                             n_events);
}

int monarch_distill_bwd(const void* dloss, const void* logits, int64_t ld, const void* teacher,
                        const void* ids, const void* labels, const void* stats, void* dlogits,
                        int64_t dld, int64_t rows, int64_t vocab, int64_t top, float temperature,
                        float mix, int dtype, void* stream, void* const* events, int n_events) {
  Distill a = {};
  a.z = logits, a.ld = ld, a.dz = dlogits, a.dld = dld, a.rows = rows;
  a.teacher = static_cast<const float*>(teacher);
  a.weight = static_cast<const float*>(dloss), a.stats_in = static_cast<const float*>(stats);
  return run_call<WITH_GRAD>(a, ids, labels, vocab, top, temperature, mix, dtype, stream, events,
                             n_events);
}

int monarch_distill_step(const void* logits, int64_t ld, const void* teacher, const void* ids,
                         const void* labels, const void* row_weight, void* loss, void* dlogits,
                         int64_t dld, int64_t rows, int64_t vocab, int64_t top, float temperature,
                         float mix, int dtype, void* stream, void* const* events, int n_events) {
  Distill a = {};
  a.z = logits, a.ld = ld, a.dz = dlogits, a.dld = dld, a.rows = rows;
  a.teacher = static_cast<const float*>(teacher);
  a.weight = static_cast<const float*>(row_weight), a.loss = static_cast<float*>(loss);
  return run_call<WITH_LOSS | WITH_GRAD>(a, ids, labels, vocab, top, temperature, mix, dtype,
                                         stream, events, n_events);
}

}  // extern "C"
