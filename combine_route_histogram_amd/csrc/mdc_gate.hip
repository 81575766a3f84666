// libmdc: routing of tokens to experts for AMD Instinct MI355X (gfx950):
// mdc_gate, whose ids and weights are the expert_ids and expert_scales of the
// dispatch and the combine.

#include "mdc_ops.h"

namespace {

// ---------------------------------------------------------------------------
// One token is handled by LPT lanes of a wavefront (16: four tokens per
// wavefront, or 64), lane l holding the scores of experts l*VPL .. +VPL in
// registers.  K rounds of "largest key" pick the experts: a maximum in the lane
// and over the lanes with DPP moves.
//
// Keys are the scores as ordered integers (order_key): integer maxima need no
// NaN rules, and INT_MIN marks an expert that is off or already taken.
//
// The choice is the one that 64-bit scores give.  A key in the rounds has the
// expert's number in its lowest bits, so that a round is one maximum: 16-bit
// logits without bias and groups fit exactly, other keys lose their lowest 8 to
// 11 bits, and probabilities are off by some rounding besides.  Rounds run once
// more than K to see the neighbour behind the last choice; where two neighbours
// are too close for such keys, a few more choices are taken and put in order by
// their scores in 64 bits, one choice a lane (gate_order); and only where that
// cannot settle it (a long run of close keys, or close groups) are all of the
// token's keys made again in 64 bits.  (Of sigmoid keys with a bias, 256 a
// token, about one token in 100 goes the second way, one in 10^5 the third.)
//
// Bound: vector instructions and the one round of wavefronts they run in.  32768
// x 256 fp32, 8 choices, is 8192 wavefronts, 8 a SIMD: 700 instructions each for
// a softmax without bias where no keys are close, 960 with sigmoid and bias, 1160
// with 4 of 8 groups as well.  At 4 cycles each that is 9, 13 and 16 us of the
// 19, 24 and 27 such launches take under the counters (23 to 25 us unprofiled;
// memory needs 5): the rest is waiting, about 5 us of it for the code of the
// second way, which few wavefronts run.  16384 x 128 bf16 take 5.8 us and 32 x 256
// 5.2 to 7.8 in a trace, where an empty kernel of as many workgroups takes 1.4 to 1.6.
// ---------------------------------------------------------------------------
constexpr int kGateThreads = 256;
constexpr float kGateLowest = -709.7827f;   // 1 / (1 + exp(-z)) of this fp32 z and below is zero in 64 bits

struct GateArgs {
  const void* logits;   // [T][E]
  const float* bias;    // [E] or NULL
  int32_t* ids;         // [T][K]
  float* weights;       // [T][K]
  int T, E, K;
  int groups, topk_groups, group_top;
  int sigmoid, renormalise;
  float scale;
  int vec;              // rows of logits (and the bias) can be read in 16-byte pieces of VPL experts
};

__device__ __forceinline__ float gate_load(const float* p) { return *p; }
__device__ __forceinline__ float gate_load(const _Float16* p) { return (float)*p; }
__device__ __forceinline__ float gate_load(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// The VPL logits of a lane, from expert `base`; -inf past the last expert.
typedef float v4f __attribute__((ext_vector_type(4)));
template <int VPL>
__device__ __forceinline__ void gate_row(const float* p, int base, const GateArgs& a, float (&z)[VPL]) {
  if constexpr (VPL % 4 == 0) {
    if (a.vec) {
#pragma unroll
      for (int j = 0; j < VPL; j += 4) {
        v4f v = {-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
        if (base < a.E) v = *reinterpret_cast<const v4f*>(p + base + j);
#pragma unroll
        for (int k = 0; k < 4; ++k) z[j + k] = v[k];
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) z[j] = base + j < a.E ? p[base + j] : -__builtin_inff();
}
template <int VPL, typename T>
__device__ __forceinline__ void gate_row(const T* p, int base, const GateArgs& a, float (&z)[VPL]) {
  if constexpr (VPL % 8 == 0) {
    if (a.vec) {
#pragma unroll
      for (int j = 0; j < VPL; j += 8) {
        v4u v = {0u, 0u, 0u, 0u};
        if (base < a.E) v = *reinterpret_cast<const v4u*>(p + base + j);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint16_t h = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
          const float f = gate_load(reinterpret_cast<const T*>(&h));
          z[j + k] = base < a.E ? f : -__builtin_inff();
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) z[j] = base + j < a.E ? gate_load(p + base + j) : -__builtin_inff();
}

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

template <typename Key>
struct GateMax {
  __device__ __forceinline__ Key operator()(Key x, Key y) const { return max(x, y); }
};
struct GateMin {
  __device__ __forceinline__ int32_t operator()(int32_t x, int32_t y) const { return min(x, y); }
};

// Keys of this lane's experts from its cleaned logits.  tol (fp32): bound on
// what a key may be off by.
template <int LPT, int VPL, typename Real>
__device__ __forceinline__ void gate_keys(const GateArgs& a, const float (&z)[VPL], int lane, float zmax,
                                          typename GateKey<Real>::type (&key)[VPL], float& tol) {
  typedef typename GateKey<Real>::type Key;
  constexpr Key kOff = GateKey<Real>::kOff;
  constexpr bool kExact = sizeof(Real) == 8;
  const int base = lane * VPL;
  tol = 0.f;
  if (a.bias == nullptr && a.groups == 1) {   // the order of the logits
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = z[j] > -__builtin_inff() ? (Key)order_key((Real)z[j]) : kOff;
    return;
  }
  Real p[VPL];
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) p[j] = gate_inv((Real)1 + gate_exp(-(Real)z[j]));
    // in 2^-24: the exponent's product 1.5 |z| s (1 - s) <= 0.34, the
    // exponential's ulp 2 s (1 - s) <= 0.5, the sum's rounding and the
    // reciprocal's ulp one each
    tol = 0x1p-22f;
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
  float b[VPL];
  if (a.bias != nullptr) gate_row<VPL>(a.bias, base, a, b);
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const Real k = a.bias == nullptr ? p[j] : p[j] + (Real)b[j];
    const bool on = z[j] > -__builtin_inff() && k > -(Real)__builtin_inff();
    key[j] = on ? order_key(k) : kOff;
    if (!kExact && on) kmax = fmaxf(kmax, fabsf((float)k));
  }
  if (!kExact) tol += 0x1p-24f * lanes_max<LPT>(fminf(kmax, 3.402823466e38f));   // the addition of the bias
}

// Whether groups of `size` experts are 1, 2, 4 .. 16 whole lanes of vpl experts.
__host__ __device__ inline bool gate_whole_lanes(int size, int vpl) {
  const int per = size / vpl;
  return size % vpl == 0 && (per & (per - 1)) == 0 && per <= 16;
}

// Turns off the keys of closed groups.  Returns whether the border between open
// and closed groups is within the scores' rounding (fp32).
template <int LPT, int VPL, typename Real>
__device__ __forceinline__ bool gate_close_groups(const GateArgs& a, int lane, float tol,
                                                  typename GateKey<Real>::type (&key)[VPL],
                                                  typename GateKey<Real>::type* lds) {
  typedef typename GateKey<Real>::type Key;
  constexpr Key kOff = GateKey<Real>::kOff;
  constexpr bool kExact = sizeof(Real) == 8;
  const int base = lane * VPL;
  const int size = a.E / a.groups;
  const int per = size / VPL;   // lanes of a group, where it is made of whole lanes
  const bool whole = gate_whole_lanes(size, VPL);
  // the group's two largest keys: in every lane of the group, or (LDS) of group g in lane g
  Key first = kOff, second = kOff;
  if (whole) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      second = max(second, min(first, key[j]));
      first = max(first, key[j]);
    }
    for (int o = 1; o < per; o <<= 1) {
      const Key f = __shfl_xor(first, o, 64), s = __shfl_xor(second, o, 64);
      second = max(max(second, s), min(first, f));
      first = max(first, f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) lds[lds_slot(base + j)] = key[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (lane < a.groups) {
      for (int i = 0; i < size; ++i) {
        const Key k = lds[lds_slot(lane * size + i)];
        second = max(second, min(first, k));
        first = max(first, k);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  auto value = [](Key k) -> Real {
    if (k == kOff) return -(Real)__builtin_inff();
    if constexpr (kExact) return __longlong_as_double(k ^ ((k >> 63) & 0x7FFFFFFFFFFFFFFFll));
    else return key_value(k);
  };
  const Real score = a.group_top == 2 ? value(first) + value(second) : value(first);
  const int group = whole ? lane / per : lane, step = whole ? per : 1;
  const bool mine = group < a.groups;
  const Key gkey = !mine ? kOff : score > -(Real)__builtin_inff() ? order_key(score) : (Key)(kOff + 1);
  int rank = 0;   // of this group among the others
  const int lane0 = threadIdx.x & 63 & ~(LPT - 1);
  for (int g = 0; g < a.groups; ++g) {
    const Key other = __shfl(gkey, lane0 + g * step, 64);
    rank += other > gkey || (other == gkey && g < group);
  }
  const bool open = mine && rank < a.topk_groups;
  bool near = false;
  if (!kExact && a.topk_groups < a.groups) {
    const int32_t lo = lanes_reduce<LPT>(open ? (int32_t)gkey : INT32_MAX, GateMin());
    const int32_t hi = lanes_reduce<LPT>(mine && !open ? (int32_t)gkey : INT32_MIN, GateMax<int32_t>());
    near = hi > (int32_t)kOff + 1 && !(key_value(lo) - key_value(hi) > 8.f * tol);   // two sums of two keys, rounded
  }
  if (whole) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = open ? key[j] : kOff;
  } else {
    const uint64_t opened = __ballot(open) >> lane0;
    const float inv = 1.0f / (float)size;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      // (e + 0.5) / size is at least 0.5 / size from a whole number: exact for e < 2048
      const int g = (int)(((float)(base + j) + 0.5f) * inv);
      if (!((opened >> (g & 63)) & 1)) key[j] = kOff;
    }
  }
  return near;
}

// Rounds on keys whose lowest bits give way to the expert's number (the lower
// number the larger key, so that equal keys go to the lowest): the id of choice
// l in lane l.  gap: what two whole keys may differ by and still be in the wrong
// order; 0: the bits given up are zero and the order is exact.  Where the first
// K are not certain, `count` choices are returned (else K), near: choices l and
// l + 1 of them may be in the wrong order.
template <int LPT, int VPL>
__device__ __forceinline__ int gate_rounds(const int32_t (&key)[VPL], int K, int lane, float gap, int& count,
                                           bool& near) {
  constexpr int kBits = LPT * VPL <= 256 ? 8 : 11;
  constexpr int32_t kNumber = (1 << kBits) - 1;
  int32_t k[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    k[j] = key[j] == INT32_MIN ? INT32_MIN : (key[j] & ~kNumber) | (kNumber - (lane * VPL + j));
  // Runs of up to four keys, largest first: a round looks at the heads and
  // moves up the run whose head it took.
  constexpr int kRun = VPL < 4 ? VPL : 4;
  auto order = [&](int i, int j) {
    const int32_t hi = max(k[i], k[j]);
    k[j] = min(k[i], k[j]);
    k[i] = hi;
  };
#pragma unroll
  for (int j = 0; j < VPL; j += kRun) {
    if constexpr (kRun > 1) order(j, j + 1);
    if constexpr (kRun > 2) {
      order(j + 2, j + 3);
      order(j, j + 2);
      order(j + 1, j + 3);
      order(j + 1, j + 2);
    }
  }
  int32_t mine = INT32_MIN, best = INT32_MIN;
  // Least distance of two keys with these upper bits (NaN behind +inf, which is near).
  auto is_near = [&](int n) {
    const int32_t below = __shfl_down(mine, 1, 64);
    const int32_t next = lane == n - 1 ? best : below;
    return lane < n && next != INT32_MIN && !(key_value(mine & ~kNumber) - key_value(next | kNumber) > gap);
  };
  near = false;
  int rounds = gap > 0.f ? K + 1 : K;
  const int more = count;
  count = K;
  for (int t = 0; t < rounds; ++t) {
    best = k[0];
#pragma unroll
    for (int j = kRun; j < VPL; j += kRun) best = max(best, k[j]);
    best = lanes_reduce<LPT>(best, GateMax<int32_t>());
#pragma unroll
    for (int j = 0; j < VPL; j += kRun) {
      const bool hit = k[j] == best;
#pragma unroll
      for (int i = 0; i < kRun; ++i) k[j + i] = !hit ? k[j + i] : i + 1 < kRun ? k[j + i + 1] : INT32_MIN;
    }
    if (t >= K) {
      near = is_near(t);
      if (t == K && __any(near)) {
        count = more;
        rounds = more + 1;
      }
    }
    mine = lane == t ? best : mine;
  }
  return mine != INT32_MIN ? kNumber - (mine & kNumber) : -1;
}

// Rounds on 64-bit keys.
template <int LPT, int VPL>
__device__ __forceinline__ int gate_rounds(int64_t (&key)[VPL], int K, int lane) {
  constexpr int64_t kOff = GateKey<double>::kOff;
  const int base = lane * VPL;
  int chosen = -1;
  for (int t = 0; t < K; ++t) {
    int64_t best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = max(best, key[j]);
    best = lanes_reduce<LPT>(best, GateMax<int64_t>());
    int32_t id = INT32_MAX;
#pragma unroll
    for (int j = VPL - 1; j >= 0; --j) id = key[j] == best ? base + j : id;
    id = lanes_reduce<LPT>(id, GateMin());
    if (best == kOff) id = -1;
    const int mine = id - base;
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = mine == j ? kOff : key[j];
    if (lane == t) chosen = id;
  }
  return chosen;
}

// Puts the first K of `count` choices (id, in lane l choice l) in the order of
// their scores in 64 bits.  A choice that is not near the one behind it is above
// all behind it.  False: all from choice K - 1 on are near, so that experts
// behind the last one would have to be looked at too.
template <int LPT, int VPL, typename T>
__device__ __forceinline__ bool gate_order(const GateArgs& a, const T* row, int lane, float zmax, int count, bool near,
                                           int& id) {
  const int lane0 = threadIdx.x & 63 & ~(LPT - 1);
  const uint64_t ends = __ballot(!near && lane >= a.K - 1 && lane < count) >> lane0;
  if (!__all((ends & (~0ull >> (64 - LPT))) != 0)) return false;
  const bool by_logit = a.bias == nullptr && a.groups == 1;
  double sum = 0;
  if (!a.sigmoid && !by_logit) {
#pragma unroll 2
    for (int j = 0; j < VPL; ++j) {
      const int e = min(lane * VPL + j, a.E - 1);
      const float z = gate_clean(gate_load(row + e));
      const double p = gate_exp((double)z - (double)zmax);
      sum += lane * VPL + j < a.E && z > -__builtin_inff() ? p : 0.0;
    }
    sum = lanes_sum<LPT>(sum);
  }
  double key = -__builtin_inf();
  if (lane < count && id >= 0) {
    const double z = gate_clean(gate_load(row + id));
    key = z;
    if (!by_logit) {
      key = a.sigmoid ? gate_inv(1.0 + gate_exp(-z)) : gate_exp(z - (double)zmax) * gate_inv(sum);
      if (a.bias != nullptr) key += (double)a.bias[id];
    }
  }
  int rank = 0;
  for (int i = 0; i < count; ++i) {
    const double other = __shfl(key, lane0 + i, 64);
    const int from = __shfl(id, lane0 + i, 64);
    rank += other > key || (other == key && from < id);
  }
  int ordered = -1;
  for (int i = 0; i < count; ++i) {
    const int there = __shfl(rank, lane0 + i, 64), from = __shfl(id, lane0 + i, 64);
    ordered = there == lane ? from : ordered;
  }
  id = ordered;
  return true;
}

// The experts of this lane's token: choice l in lane l < K, -1 for none.
template <int LPT, int VPL, typename T>
__device__ __forceinline__ int gate_pick(const GateArgs& a, const T* row, const float (&z)[VPL], int lane, float zmax,
                                         int64_t* lds) {
  int32_t key[VPL];
  float tol;
  gate_keys<LPT, VPL, float>(a, z, lane, zmax, key, tol);
  bool border = false;
  if (a.groups > 1) border = gate_close_groups<LPT, VPL, float>(a, lane, tol, key, reinterpret_cast<int32_t*>(lds));
  if (!__any(border)) {
    const bool by_logit = a.bias == nullptr && a.groups == 1;
    // (fp16's 11 significant bits leave 13 of fp32's free, bf16's 16; fp32 logits are equal or a step apart)
    const float gap = !by_logit ? 2.f * tol : sizeof(T) == 2 ? 0.f : 0x1p-149f;
    int count = min(a.K + 4, LPT);
    bool near;
    int id = gate_rounds<LPT, VPL>(key, a.K, lane, gap, count, near);
    if (!__any(near && lane < a.K)) return id;
    if (gate_order<LPT, VPL>(a, row, lane, zmax, count, near, id)) return id;
  }
  int64_t key64[VPL];
  float none;
  gate_keys<LPT, VPL, double>(a, z, lane, zmax, key64, none);
  if (a.groups > 1) (void)gate_close_groups<LPT, VPL, double>(a, lane, 0.f, key64, lds);
  return gate_rounds<LPT, VPL>(key64, a.K, lane);
}

template <typename T, int LPT, int VPL>
__global__ __launch_bounds__(kGateThreads) void k_gate(GateArgs a) {
  extern __shared__ int64_t gate_lds[];
  constexpr int kTokens = kGateThreads / LPT;
  const int lane = threadIdx.x & (LPT - 1);
  const int slot = threadIdx.x / LPT;
  const int64_t token = grid_block() * kTokens + slot;
  const int64_t t = min(token, (int64_t)a.T - 1);   // (lanes past the last token repeat it and store nothing)
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  const int base = lane * VPL;
  float z[VPL];
  gate_row<VPL>(row, base, a, z);
  float zmax = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    z[j] = gate_clean(z[j]);
    zmax = fmaxf(zmax, z[j]);
  }
  if (!a.sigmoid) zmax = lanes_max<LPT>(zmax);
  int64_t* lds = gate_lds + (int64_t)slot * (LPT * VPL + (LPT * VPL >> 5));
  const int id = gate_pick<LPT, VPL>(a, row, z, lane, zmax, lds);

  // Weights from the logits of the chosen experts, choice k in lane k.
  const bool have = lane < a.K && id >= 0;
  const float zc = have ? gate_clean(gate_load(row + id)) : -__builtin_inff();
  float w = 0.f;
  if (a.sigmoid) {
    w = have ? 1.0f / (1.0f + expf(-zc)) : 0.f;
    if (a.renormalise) {
      // Scores of logits below -87 leave fp32, their quotients do not: where the
      // largest chosen logit is negative, every score is divided by its
      // exponential.  (A score is zero where it is in 64 bits, whose exp(-z)
      // ends at z = -709.78.)
      const float top = lanes_max<LPT>(zc);
      if (top < 0.f) w = zc > kGateLowest ? expf(zc - top) / (1.0f + expf(zc)) : 0.f;
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
    a.ids[token * a.K + lane] = id;
    a.weights[token * a.K + lane] = w * a.scale;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <typename T, int LPT, int VPL>
void launch_gate(GateArgs a, hipStream_t s) {
  a.vec = a.E % VPL == 0 && a.E * sizeof(T) % 16 == 0 && aligned16(a.logits) && aligned16(a.bias);
  constexpr int kTokens = kGateThreads / LPT;
  const size_t lds = a.groups > 1 && !gate_whole_lanes(a.E / a.groups, VPL) ? (size_t)kTokens * lds_slots(LPT, VPL) * sizeof(int64_t) : 0;
  hipLaunchKernelGGL((k_gate<T, LPT, VPL>), grid_of(((int64_t)a.T + kTokens - 1) / kTokens), dim3(kGateThreads), lds, s, a);
}

template <typename T>
void launch_gate_typed(const GateArgs& a, hipStream_t s) {
  // Four tokens per wavefront where there are enough of them to fill the chip
  // that way; else, or where a token's experts need more registers than that
  // leaves, a wavefront per token.  Sigmoid with bias, four tokens : one token, in
  // us: 64 experts 6.6 : 6.7 at 2048 tokens, 6.7 : 7.5 at 4096, 8.1 : 13.3 at
  // 16384; 256 experts in 8 groups 9.7 : 8.4, 9.9 : 9.9 and 16.6 : 20.8.
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
                   p.group_top, p.score == MDC_GATE_SIGMOID, p.renormalise, p.scale, 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.dtype == MDC_DTYPE_BF16) launch_gate_typed<uint16_t>(a, s);
  else if (p.dtype == MDC_DTYPE_FP16) launch_gate_typed<_Float16>(a, s);
  else launch_gate_typed<float>(a, s);
  return launched();
}

}  // extern "C"
