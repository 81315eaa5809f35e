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
// A team of threads takes a row. Exponentials are 2^((z - m) log2(e) / T) with m
// the row's maximum: z - m is exact or rounded once, and rows of the type's
// lowest value (m huge) stay finite. Sums are fp32.
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

enum { WITH_LOSS = 1, WITH_GRAD = 2 };   // loss and sums from z; gradient

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum and sums of exponentials of one thread's share of a row.
struct Running {
  float m = -3.402823466e38f, st = 0.0f, s1 = 0.0f;
  template <bool TWO, int N>
  __device__ __forceinline__ void add(const float (&v)[N], float ct) {
    float pm = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) pm = fmaxf(pm, v[i]);
    if (pm > m) {
      st *= exp2_of((m - pm) * ct);
      if constexpr (TWO) s1 *= exp2_of((m - pm) * kLog2e);
      m = pm;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      st += exp2_of((v[i] - m) * ct);
      if constexpr (TWO) s1 += exp2_of((v[i] - m) * kLog2e);
    }
  }
};

// a row's piece as fp32, -inf past its end
template <typename T, int N>
__device__ __forceinline__ void unpack_row(const u32x4& r, int at, int d, float (&v)[N]) {
  PieceOf<T>::unpack(r, v);
  if (at + N > d)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at + i >= d) v[i] = -INFINITY;
}

// TWO: a second sum at temperature 1 (a label term whose softmax is not q).
template <typename T, int TEAM, int WHAT, bool TWO>
__global__ __launch_bounds__(TEAM) void distill_kernel(Distill a) {
  constexpr int N = PieceOf<T>::N, U = 4;
  __shared__ typename Team<TEAM>::Lds tlds;
  __shared__ int s_id[MONARCH_DISTILL_MAX_TOP];
  __shared__ float s_p[MONARCH_DISTILL_MAX_TOP], s_z[MONARCH_DISTILL_MAX_TOP];
  Team<TEAM> team(&tlds);
  const int tid = threadIdx.x;
  const float ct = kLog2e / a.temperature;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + row * a.ld;
    // the teacher's entries and the student's logits there
    float tmax = -INFINITY;
    for (int k = tid; k < a.top; k += TEAM) {
      const int64_t id = a.ids[row * a.top + k];
      const float t = a.teacher[row * a.top + k];
      const bool ok = id >= 0 && id < a.vocab && t > -INFINITY;
      s_id[k] = ok ? static_cast<int>(id) : -1;
      s_p[k] = t;
      s_z[k] = ok ? Io<T>::load(z, id) : 0.0f;
      if (ok) tmax = fmaxf(tmax, t);
    }
    const int64_t label = a.labels ? a.labels[row] : -1;
    const bool told = label >= 0 && label < a.vocab && a.mix < 1.0f;
    const float zl = told ? Io<T>::load(z, label) : 0.0f;

    float red[3];
    float m, st = 0.0f, s1 = 0.0f;
    if constexpr (WHAT & WITH_LOSS) {
      Running r;
      for (int base = 0; base < a.vocab; base += TEAM * N * U) {
        u32x4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = base + (u * TEAM + tid) * N;
          if (at < a.vocab) raw[u] = load_piece<T, true>(z, at, a.vocab);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = base + (u * TEAM + tid) * N;
          if (at < a.vocab) {
            float v[N];
            unpack_row<T, N>(raw[u], at, a.vocab, v);
            r.template add<TWO, N>(v, ct);
          }
        }
      }
      red[0] = r.m;
      red[1] = tmax;
      team.template reduce<MaxOp, 2>(*reinterpret_cast<float(*)[2]>(red));
      m = red[0];
      tmax = red[1];
      st = r.st * exp2_of((r.m - m) * ct);
      s1 = TWO ? r.s1 * exp2_of((r.m - m) * kLog2e) : 0.0f;
    } else {
      red[0] = tmax;
      team.template reduce<MaxOp, 1>(*reinterpret_cast<float(*)[1]>(red));
      tmax = red[0];
      m = a.stats_in[row * 4];
    }
    const bool some = tmax > -INFINITY && a.mix > 0.0f;
    float tsum = 0.0f;
    for (int k = tid; k < a.top; k += TEAM)
      if (s_id[k] >= 0) {
        const float e = exp2_of((s_p[k] - tmax) * ct);
        s_p[k] = e;
        tsum += e;
      } else {
        s_p[k] = 0.0f;
      }
    red[0] = tsum;
    red[1] = st;
    red[2] = s1;
    if constexpr (WHAT & WITH_LOSS) {
      team.template reduce<SumOp, 3>(red);
      st = red[1];
      s1 = TWO ? red[2] : st;
    } else {
      team.template reduce<SumOp, 1>(*reinterpret_cast<float(*)[1]>(red));
      st = a.stats_in[row * 4 + 1];
      s1 = a.stats_in[row * 4 + 2];
    }
    const float inv_t = some ? 1.0f / red[0] : 0.0f;
    const bool alive = st != 0.0f;   // NaN counts as alive: it has to come out
    if constexpr (WHAT & WITH_LOSS) {
      // T (log p_k - log q_k) = (t_k - tmax) - (z_k - m) + T (log st - log tsum): not
      // divided by T, so that a logit of the type's lowest value does not overflow
      float kl = 0.0f;
      if (some && alive) {
        const float base = a.temperature * (logf(st) - logf(red[0]));
        for (int k = tid; k < a.top; k += TEAM) {
          const float p = s_p[k] * inv_t;
          if (p > 0.0f) {
            const float t = a.teacher[row * a.top + k];
            kl = fmaf(p, (t - tmax) - (s_z[k] - m) + base, kl);
          } else if (p != p) {
            kl = p;
          }
        }
      }
      kl = team.sum(kl);
      if (tid == 0) {
        float loss = a.mix * a.temperature * kl;
        if (told && alive) loss += (1.0f - a.mix) * (logf(s1) - (zl - m));
        if (!some && !told) loss = 0.0f;
        a.loss[row] = loss;
        if (a.stats) *reinterpret_cast<f32x4*>(a.stats + row * 4) = f32x4{m, st, s1, 0.0f};
      }
    }
    if constexpr (WHAT & WITH_GRAD) {
      const float w = a.weight ? a.weight[row] : 1.0f;
      const float ga = some && alive ? w * a.mix * a.temperature : 0.0f;
      const float gb = told && alive ? w * (1.0f - a.mix) : 0.0f;
      // one softmax for both terms where they share it
      const float fa = TWO ? ga / st : (ga + gb) / st, fb = TWO ? gb / s1 : 0.0f;
      T* dz = static_cast<T*>(a.dz) + row * a.dld;
      const bool nothing = (!some && !told) || !alive;
      auto grad = [&](float v) {
        float g = fa * exp2_of((v - m) * ct);
        if constexpr (TWO) g = fmaf(fb, exp2_of((v - m) * kLog2e), g);
        return g;
      };
      for (int base = 0; base < a.vocab; base += TEAM * N * U) {
        u32x4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = base + (u * TEAM + tid) * N;
          if (at < a.vocab) raw[u] = load_piece<T, true>(z, at, a.vocab);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = base + (u * TEAM + tid) * N;
          if (at < a.vocab) {
            float v[N];
            PieceOf<T>::unpack(raw[u], v);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = nothing ? 0.0f : grad(v[i]);
            store_piece<T, true>(dz, at, a.vocab, PieceOf<T>::pack(v));
          }
        }
      }
      // the entries and the label: their elements are written again, whole
      __syncthreads();
      if (!nothing) {
        for (int k = tid; k < a.top; k += TEAM) {
          const int id = s_id[k];
          if (id < 0) continue;
          float p = 0.0f;
          bool first = true;
          for (int j = 0; j < a.top; ++j)
            if (s_id[j] == id) {
              p += s_p[j];
              first = first && j >= k;
            }
          if (!first) continue;
          float g = grad(s_z[k]) - ga * (p * inv_t);
          if (told && id == label) g -= gb;
          Io<T>::store(dz, id, g);
        }
        if (told) {
          int hit = 0;
          for (int k = tid; k < a.top; k += TEAM) hit |= s_id[k] == label;
          hit = __syncthreads_or(hit);
          if (!hit && tid == 0) Io<T>::store(dz, label, grad(zl) - gb);
        }
      }
    }
    __syncthreads();   // the next row overwrites the entries
  }
}

int check_sizes(int64_t rows, int64_t vocab, int64_t ld, int64_t top, int dtype) {
  if (dtype != MONARCH_F32 && dtype != MONARCH_BF16) return MONARCH_ERR_DTYPE;
  if (rows < 0 || rows >= kLimit || vocab <= 0 || vocab >= kLimit || ld < vocab || top < 0 ||
      top > MONARCH_DISTILL_MAX_TOP)
    return MONARCH_ERR_SHAPE;
  return MONARCH_OK;
}

bool off_elements(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) != 0;
}

template <typename T, int TEAM, int WHAT>
hipError_t launch_two(const Distill& a, bool two, hipStream_t s) {
  const int64_t grid = a.rows < (1 << 20) ? a.rows : (1 << 20);
  if (two)
    hipLaunchKernelGGL((distill_kernel<T, TEAM, WHAT, true>), dim3(static_cast<unsigned>(grid)),
                       dim3(TEAM), 0, s, a);
  else
    hipLaunchKernelGGL((distill_kernel<T, TEAM, WHAT, false>), dim3(static_cast<unsigned>(grid)),
                       dim3(TEAM), 0, s, a);
  return hipGetLastError();
}

template <int WHAT>
hipError_t launch(const Distill& a, bool bf16, hipStream_t s) {
  const bool two = a.labels && a.mix < 1.0f && a.temperature != 1.0f;
  if (bf16) return launch_two<uint16_t, 512, WHAT>(a, two, s);
  return launch_two<float, 512, WHAT>(a, two, s);
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
