// libmdc: routing of tokens to experts for AMD Instinct MI355X (gfx950):
// mdc_gate, whose ids and weights are the expert_ids and expert_scales of the
// dispatch and the combine.

#include "mdc_common.h"

namespace {

// ---------------------------------------------------------------------------
// One token is handled by LPT lanes of a wavefront (16: four tokens per
// wavefront, or 64), lane l holding the scores of experts l*VPL .. +VPL in
// registers.  K rounds of "largest key, lowest index" pick the experts: a
// maximum and an index minimum over the LPT lanes with DPP moves.
//
// Keys are the scores as ordered integers (order_key): integer maxima need no
// NaN rules, and INT_MIN marks an expert that is off or already taken.
//
// The choice is the one that exact scores give.  Keys made of probabilities
// are rounded, so the fp32 rounds run once more than K and compare neighbours:
// when two keys closer than their error bound might be in the wrong order (and
// are not equal by equal inputs), the wavefront repeats its tokens with 64-bit
// scores.  Without a bias and groups the key is the logit itself, exact.
// ---------------------------------------------------------------------------
constexpr int kGateThreads = 256;

struct GateArgs {
  const void* logits;   // [T][E]
  const float* bias;    // [E] or NULL
  int32_t* ids;         // [T][K]
  float* weights;       // [T][K]
  int T, E, K;
  int groups, topk_groups, group_top;
  int sigmoid, renormalise;
  float scale;
};

__device__ __forceinline__ float gate_load(const float* p) { return *p; }
__device__ __forceinline__ float gate_load(const _Float16* p) { return (float)*p; }
__device__ __forceinline__ float gate_load(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// NaN -> -inf (the expert is off), +inf -> the largest finite value.
__device__ __forceinline__ float gate_clean(float z) {
  return z > -__builtin_inff() ? fminf(z, 3.402823466e38f) : -__builtin_inff();
}

// Floating values as integers of the same order; -0 counts as +0.
__device__ __forceinline__ int32_t order_key(float v) {
  const int32_t b = __float_as_int(v + 0.0f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ int64_t order_key(double v) {
  const int64_t b = __double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFFll);
}
__device__ __forceinline__ float key_value(int32_t k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

template <typename Real>
struct GateKey;
template <>
struct GateKey<float> {
  typedef int32_t type;
  static constexpr int32_t kOff = INT32_MIN;
};
template <>
struct GateKey<double> {
  typedef int64_t type;
  static constexpr int64_t kOff = INT64_MIN;
};

// Value of the lane that differs in the given way, for reductions over the
// 16 lanes of a DPP row (xor 1, xor 2, half mirror, mirror) and over the rows.
template <int CTRL>
__device__ __forceinline__ int32_t dpp(int32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}

// op over the LPT lanes of a token; every lane receives the result.
template <int LPT, typename F>
__device__ __forceinline__ int32_t lanes_reduce(int32_t v, F op) {
  v = op(v, dpp<0xB1>(v));
  v = op(v, dpp<0x4E>(v));
  v = op(v, dpp<0x141>(v));
  v = op(v, dpp<0x140>(v));
  if (LPT == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false);
    v = op((int32_t)a[0], (int32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap((unsigned)v, (unsigned)v, false, false);
    v = op((int32_t)b[0], (int32_t)b[1]);
  }
  return v;
}
template <int LPT, typename F>
__device__ __forceinline__ int64_t lanes_reduce(int64_t v, F op) {
#pragma unroll
  for (int o = 1; o < LPT; o <<= 1) v = op(v, __shfl_xor(v, o, 64));
  return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
  return __int_as_float(lanes_reduce<LPT>(
      __float_as_int(v), [](int32_t a, int32_t b) { return __float_as_int(__int_as_float(a) + __int_as_float(b)); }));
}
template <int LPT>
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int o = 1; o < LPT; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  return key_value(lanes_reduce<LPT>(order_key(v), [](int32_t a, int32_t b) { return max(a, b); }));
}

__device__ __forceinline__ float gate_exp(float v) { return __expf(v); }
__device__ __forceinline__ double gate_exp(double v) { return exp(v); }
__device__ __forceinline__ float gate_inv(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ double gate_inv(double v) { return 1.0 / v; }

// Keys of one token in LDS: expert e at e + e / 32, so that lanes which walk
// groups of 32 or 64 experts side by side read different banks.
__device__ __forceinline__ int lds_slot(int e) { return e + (e >> 5); }
inline int lds_slots(int lpt, int vpl) { return lpt * vpl + (lpt * vpl >> 5); }

// What a token's lanes know after the rounds.
struct GatePick {
  int id, next_id;   // lane l < K: expert of choice l, and of choice l + 1 (-1: none)
  bool near;         // the order of two keys is within their rounding
};

// Chooses the K experts of this lane's token from its cleaned logits.  near is
// only looked for in fp32.
template <int LPT, int VPL, typename Real>
__device__ __forceinline__ GatePick gate_pick(const GateArgs& a, const float (&z)[VPL], int lane, float zmax,
                                              typename GateKey<Real>::type* lds) {
  typedef typename GateKey<Real>::type Key;
  constexpr Key kOff = GateKey<Real>::kOff;
  constexpr bool kExact = sizeof(Real) == 8;
  const int base = lane * VPL;
  const bool by_logit = a.bias == nullptr && a.groups == 1;
  Key key[VPL];
  float tol = 0.f;   // bound on what two keys' difference may be off by (fp32)
  if (by_logit) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = z[j] > -__builtin_inff() ? (Key)order_key((Real)z[j]) : kOff;
  } else {
    Real p[VPL];
    if (a.sigmoid) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) p[j] = gate_inv((Real)1 + gate_exp(-(Real)z[j]));
      // exp, sum and reciprocal: s (1 - s) |z| 2^-23 + 2 ulp of s, below 2^-22 each
      tol = 0x1p-20f;
    } else {
      Real sum = 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        p[j] = z[j] > -__builtin_inff() ? gate_exp((Real)z[j] - (Real)zmax) : (Real)0;
        sum += p[j];
      }
      sum = lanes_sum<LPT>(sum);
      const Real inv = gate_inv(sum);   // (no expert live: infinite, and no key uses it)
#pragma unroll
      for (int j = 0; j < VPL; ++j) p[j] *= inv;
      // the sum's relative error (VPL + 6 additions) and the exponentials'
      // reach every key in proportion to its probability, at most 1 / sum
      tol = 0x1p-17f * (float)inv;
    }
    float kmax = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const Real k = a.bias == nullptr ? p[j] : p[j] + (Real)(base + j < a.E ? a.bias[base + j] : 0.f);
      const bool on = z[j] > -__builtin_inff() && k > -(Real)__builtin_inff();
      key[j] = on ? order_key(k) : kOff;
      if (!kExact && on) kmax = fmaxf(kmax, fabsf((float)k));
    }
    if (!kExact) tol += 0x1p-22f * lanes_max<LPT>(fminf(kmax, 3.402823466e38f));   // the additions of the bias
  }
  GatePick r{-1, -1, false};
  if (a.groups > 1) {
    // lane g scans group g's keys in LDS for its group_top largest
    const int size = a.E / a.groups;
#pragma unroll
    for (int j = 0; j < VPL; ++j) lds[lds_slot(base + j)] = key[j];
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    Key first = kOff, second = kOff;
    const bool mine = lane < a.groups;
    if (mine) {
      for (int i = 0; i < size; ++i) {
        const Key k = lds[lds_slot(lane * size + i)];
        second = max(second, min(first, k));
        first = max(first, k);
      }
    }
    auto value = [](Key k) -> Real {
      if (k == kOff) return -(Real)__builtin_inff();
      if constexpr (kExact) {
        return __longlong_as_double(k ^ ((k >> 63) & 0x7FFFFFFFFFFFFFFFll));
      } else {
        return key_value(k);
      }
    };
    const Real score = a.group_top == 2 ? value(first) + value(second) : value(first);
    const Key gkey = !mine ? kOff : score > -(Real)__builtin_inff() ? order_key(score) : (Key)(kOff + 1);
    // rank of each group among the others
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const Key other = __shfl(gkey, (threadIdx.x & 63 & ~(LPT - 1)) + g, 64);
      rank += other > gkey || (other == gkey && g < lane);
    }
    const bool open = mine && rank < a.topk_groups;
    if (!kExact && a.topk_groups < a.groups) {
      auto least = [](int32_t x, int32_t y) { return min(x, y); };
      auto most = [](int32_t x, int32_t y) { return max(x, y); };
      const int32_t lo = lanes_reduce<LPT>(open ? (int32_t)gkey : INT32_MAX, least);
      const int32_t hi = lanes_reduce<LPT>(mine && !open ? (int32_t)gkey : INT32_MIN, most);
      r.near = hi > kOff + 1 && !(key_value(lo) - key_value(hi) > 3.f * tol);   // a sum of two keys
    }
    const uint64_t opened = __ballot(open) >> (threadIdx.x & 63 & ~(LPT - 1));
    const float per = 1.0f / (float)size;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      // (e + 0.5) / size is at least 0.5 / size from a whole number: exact for e < 2048
      const int g = (int)(((float)(base + j) + 0.5f) * per);
      if (!((opened >> (g & 63)) & 1)) key[j] = kOff;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  const int rounds = by_logit || kExact ? a.K : a.K + 1;
  Key prev = kOff;
  for (int k = 0; k < rounds; ++k) {
    Key best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = max(best, key[j]);
    best = lanes_reduce<LPT>(best, [](Key x, Key y) { return max(x, y); });
    if (__all(best == kOff)) break;   // (of this wavefront's tokens)
    int32_t id = INT32_MAX;
#pragma unroll
    for (int j = VPL - 1; j >= 0; --j) id = key[j] == best ? base + j : id;
    id = lanes_reduce<LPT>(id, [](int32_t x, int32_t y) { return min(x, y); });
    if (best == kOff) id = -1;
    const int mine = id - base;
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = mine == j ? kOff : key[j];
    if (lane == k) r.id = id;
    if (!kExact && !by_logit) {
      if (lane == k - 1) {
        r.next_id = id;
        r.near |= id >= 0 && !(key_value((int32_t)prev) - key_value((int32_t)best) > 2.f * tol);
      }
      prev = best;
    }
  }
  return r;
}

template <typename T, int LPT, int VPL>
__global__ __launch_bounds__(kGateThreads) void k_gate(GateArgs a) {
  extern __shared__ int64_t gate_lds[];
  constexpr int kTokens = kGateThreads / LPT;
  const int lane = threadIdx.x & (LPT - 1);
  const int slot = threadIdx.x / LPT;
  const int token = blockIdx.x * kTokens + slot;
  const int t = min(token, a.T - 1);   // (lanes past the last token repeat it and store nothing)
  const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.E;
  const int base = lane * VPL;
  float z[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) z[j] = base + j < a.E ? gate_load(row + base + j) : -__builtin_inff();
  float zmax = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    z[j] = gate_clean(z[j]);
    zmax = fmaxf(zmax, z[j]);
  }
  if (!a.sigmoid) zmax = lanes_max<LPT>(zmax);
  int64_t* lds = gate_lds + (int64_t)slot * (LPT * VPL + (LPT * VPL >> 5));
  GatePick r = gate_pick<LPT, VPL, float>(a, z, lane, zmax, reinterpret_cast<int32_t*>(lds));
  if (r.near && r.id >= 0 && r.next_id >= 0 && a.groups == 1) {
    // equal inputs have equal keys: their order by index is right
    r.near = !(gate_load(row + r.id) == gate_load(row + r.next_id) &&
               (a.bias == nullptr || a.bias[r.id] == a.bias[r.next_id]));
  }
  if (__any(r.near)) r = gate_pick<LPT, VPL, double>(a, z, lane, zmax, lds);

  // Weights from the logits of the chosen experts, choice k in lane k.
  const bool have = lane < a.K && r.id >= 0;
  const float zc = have ? gate_clean(gate_load(row + r.id)) : -__builtin_inff();
  float w = 0.f;
  if (a.sigmoid) {
    w = have ? 1.0f / (1.0f + expf(-zc)) : 0.f;
    if (a.renormalise) {
      const float sum = lanes_sum<LPT>(w);
      w = sum > 0.f ? w / sum : 0.f;
    }
  } else if (a.renormalise) {
    // the softmax over the chosen experts: the sum over all of them cancels
    const float top = lanes_max<LPT>(zc);
    w = have ? expf(zc - top) : 0.f;
    const float sum = lanes_sum<LPT>(w);
    w = have ? w / sum : 0.f;
  } else {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum += z[j] > -__builtin_inff() ? __expf(z[j] - zmax) : 0.f;
    sum = lanes_sum<LPT>(sum);
    w = have ? expf(zc - zmax) / sum : 0.f;
  }
  if (lane < a.K && token < a.T) {
    a.ids[(int64_t)token * a.K + lane] = r.id;
    a.weights[(int64_t)token * a.K + lane] = w * a.scale;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <typename T, int LPT, int VPL>
void launch_gate(const GateArgs& a, hipStream_t s) {
  constexpr int kTokens = kGateThreads / LPT;
  const size_t lds = a.groups > 1 ? (size_t)kTokens * lds_slots(LPT, VPL) * sizeof(int64_t) : 0;
  hipLaunchKernelGGL((k_gate<T, LPT, VPL>), dim3((a.T + kTokens - 1) / kTokens), dim3(kGateThreads), lds, s, a);
}

template <typename T>
void launch_gate_typed(const GateArgs& a, hipStream_t s) {
  // Four tokens per wavefront where there are enough of them to fill the chip
  // that way; else, or where a token's experts need more registers than that
  // leaves, a wavefront per token.
  const bool four = a.T >= 4096 && a.E <= 256 && a.groups <= 16;
  if (four && a.E <= 64) launch_gate<T, 16, 4>(a, s);
  else if (four && a.E <= 128) launch_gate<T, 16, 8>(a, s);
  else if (four) launch_gate<T, 16, 16>(a, s);
  else if (a.E <= 64) launch_gate<T, 64, 1>(a, s);
  else if (a.E <= 128) launch_gate<T, 64, 2>(a, s);
  else if (a.E <= 256) launch_gate<T, 64, 4>(a, s);
  else if (a.E <= 512) launch_gate<T, 64, 8>(a, s);
  else if (a.E <= 1024) launch_gate<T, 64, 16>(a, s);
  else launch_gate<T, 64, 32>(a, s);
}

}  // namespace

extern "C" {

mdc_status mdc_gate(const mdc_shape* shape, const mdc_gate_params* params, const void* logits, const float* bias,
                    int32_t* expert_ids, float* expert_scales, void* stream) {
  const mdc_status st = check_shape(shape);
  if (st != MDC_OK) return st;
  if (params == nullptr) return MDC_ERR_NULLPTR;
  const int64_t E = (int64_t)shape->num_experts + shape->zero_experts + shape->copy_experts;
  const mdc_gate_params& p = *params;
  if (p.dtype < MDC_DTYPE_BF16 || p.dtype > MDC_DTYPE_FP32) return MDC_ERR_INVALID;
  if (p.score != MDC_GATE_SOFTMAX && p.score != MDC_GATE_SIGMOID) return MDC_ERR_INVALID;
  if (p.groups < 1 || E % p.groups != 0 || p.topk_groups < 1 || p.topk_groups > p.groups) return MDC_ERR_INVALID;
  if (p.group_top < 1 || p.group_top > 2 || p.group_top > E / p.groups) return MDC_ERR_INVALID;
  if (shape->topk > E / p.groups * p.topk_groups) return MDC_ERR_INVALID;
  if (p.renormalise != 0 && p.renormalise != 1) return MDC_ERR_INVALID;
  if (!(p.scale - p.scale == 0.f)) return MDC_ERR_INVALID;   // infinite or NaN
  if (E > MDC_MAX_GATE_EXPERTS || p.groups > MDC_MAX_GATE_GROUPS) return MDC_ERR_UNSUPPORTED;
  const int64_t T = (int64_t)shape->world * shape->bs;
  if (T == 0) return MDC_OK;
  if (logits == nullptr || expert_ids == nullptr || expert_scales == nullptr) return MDC_ERR_NULLPTR;
  const uintptr_t size = p.dtype == MDC_DTYPE_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size != 0 || !aligned4(bias) || !aligned4(expert_ids) ||
      !aligned4(expert_scales))
    return MDC_ERR_INVALID;
  const GateArgs a{logits, bias, expert_ids, expert_scales, (int)T, (int)E, shape->topk, p.groups, p.topk_groups,
                   p.group_top, p.score == MDC_GATE_SIGMOID, p.renormalise, p.scale};
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.dtype == MDC_DTYPE_BF16) launch_gate_typed<uint16_t>(a, s);
  else if (p.dtype == MDC_DTYPE_FP16) launch_gate_typed<_Float16>(a, s);
  else launch_gate_typed<float>(a, s);
  return launched();
}

}  // extern "C"
