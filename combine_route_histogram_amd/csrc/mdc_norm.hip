// libmdc: residual addition and RMS norm with 16-bit and 8-bit outputs for
// AMD Instinct MI355X (gfx950): mdc_add_rms_norm.

#include "mdc_fp8.h"

namespace {

// ---------------------------------------------------------------------------
// One workgroup per row, the row in registers (VPT vectors of 8 elements per
// thread, vector u of thread t at t + u * threads): x and the residual are
// read once, and everything the row gives is written from registers.  The sum
// of squares is per-thread fp32 sums, then DPP adds and one LDS exchange.
// Sixteen consecutive lanes hold one 128-column run, so an fp8 scale is a
// maximum over a DPP row; the int8 row scale takes a second LDS exchange.
//
// Sums and everything up to the outputs are fp32; residual_out, y and q are
// rounded once each, from the unrounded values.
//
// Bound: memory.  16384 rows of 7168 (bf16, residual in and out, y, fp8 rows
// and scales: 1.06 GB) 184 us, 5.8 TB/s, where a plain read and a plain write of
// its bytes take 172; 2051 x 5000 (fp16, fp32 residual, int8 out) 23 us, 4.9 TB/s;
// 32 x 7168 3.8 us, of which an empty launch takes 1.4 and trips to memory the rest.
// ---------------------------------------------------------------------------
struct NormArgs {
  const void* x;
  const void* res;       // or NULL
  const void* weight;
  void* res_out;         // or NULL
  void* y;               // or NULL
  void* q;               // or NULL
  float* q_scale;
  int rows, nvec;        // vectors of 8 elements per row
  float eps, inv_hidden;
};

struct Bf16 {
  uint16_t bits;
};

// Eight elements from and to memory.
__device__ __forceinline__ void load8(const Bf16* p, float (&v)[8]) {
  const v4u w = *reinterpret_cast<const v4u*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v8f __attribute__((ext_vector_type(8)));
__device__ __forceinline__ void load8(const _Float16* p, float (&v)[8]) {
  const v8h w = *reinterpret_cast<const v8h*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)w[i];
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const v4f a = reinterpret_cast<const v4f*>(p)[0], b = reinterpret_cast<const v4f*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ void store8(Bf16* p, const float (&v)[8]) {
  v8f f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = v[i];
  *reinterpret_cast<v8b*>(p) = __builtin_convertvector(f, v8b);   // nearest, ties to even
}
__device__ __forceinline__ void store8(_Float16* p, const float (&v)[8]) {
  v8h w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = (_Float16)v[i];
  *reinterpret_cast<v8h*>(p) = w;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<v4f*>(p)[0] = v4f{v[0], v[1], v[2], v[3]};
  reinterpret_cast<v4f*>(p)[1] = v4f{v[4], v[5], v[6], v[7]};
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

constexpr int kNormThreads = 1024;   // most threads of a workgroup

template <typename T, typename R, typename Wt, int QUANT, int VPT>
__global__ __launch_bounds__(kNormThreads) void k_add_rms_norm(NormArgs a) {
  __shared__ float part[kNormThreads / 64];
  __shared__ uint32_t part_max[kNormThreads / 64];
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
  const int64_t row = grid_block();
  if (row >= a.rows) return;
  const int64_t at = row * a.nvec;   // first vector of the row
  float h[VPT][8];
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = tid + u * threads;
    if (i < a.nvec) {
      load8(static_cast<const T*>(a.x) + (at + i) * 8, h[u]);
      if (a.res != nullptr) {
        float r[8];
        load8(static_cast<const R*>(a.res) + (at + i) * 8, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[u][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[u][j], h[u][j], sum);
  }
  sum = wave_sum(sum);
  if ((tid & 63) == 0) part[tid >> 6] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < waves; ++w) sum += part[w];
  const float inv = 1.0f / sqrtf(sum * a.inv_hidden + a.eps);
  uint32_t amax = 0;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = tid + u * threads;
    float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // h * weight, v before the row's factor
    if (i < a.nvec) {
      if (a.res_out != nullptr) store8(static_cast<R*>(a.res_out) + (at + i) * 8, h[u]);
      float w[8];
      load8(static_cast<const Wt*>(a.weight) + i * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (QUANT == MDC_QUANT_FP8) t[j] = h[u][j] * w[j];
        h[u][j] = h[u][j] * inv * w[j];   // (h times a large or tiny weight may leave fp32)
      }
      if (a.y != nullptr) store8(static_cast<T*>(a.y) + (at + i) * 8, h[u]);
    }
    uint32_t m = 0;
    if (QUANT != MDC_QUANT_NONE)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(QUANT == MDC_QUANT_FP8 ? t[j] : h[u][j]));
    if (QUANT == MDC_QUANT_FP8) {
      // The row's factor is in v and in amax alike, so the codes are those of
      // t, a rounding nearer (often all of 16-bit values' product); of v where
      // t or v leaves the ordinary range (for all 16 lanes of a run or none).
      m = row16_max(m);
      const float top = __uint_as_float(m) * inv;
      const bool plain = __uint_as_float(m) >= 0x1p-100f && top >= kFp8AmaxMin && top < __builtin_inff();
      if (!plain) {
        m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          t[j] = h[u][j];
          m = max(m, abs_bits(t[j]));
        }
        m = row16_max(m);
      }
      Fp8Scaler s(m);
      if (plain) s.scale = top / kFp8Max;
      if (i < a.nvec) {
        reinterpret_cast<uint2*>(a.q)[at + i] = uint2{s.codes4(t[0], t[1], t[2], t[3]),
                                                      s.codes4(t[4], t[5], t[6], t[7])};
        if ((i & 15) == 0) a.q_scale[row * ((a.nvec + 15) >> 4) + (i >> 4)] = s.scale;
      }
    }
    amax = max(amax, m);
  }
  if (QUANT == MDC_QUANT_INT8) {
    amax = wave_max(amax);
    if ((tid & 63) == 0) part_max[tid >> 6] = amax;
    __syncthreads();
    amax = 0;
    for (int w = 0; w < waves; ++w) amax = max(amax, part_max[w]);
    const float top = __uint_as_float(amax);
    float scale = amax != 0 ? 127.0f / top : 0.f;
    if (scale > 3.402823466e38f) scale = 3.402823466e38f;   // (infinite, it would make NaN of the row's zeros)
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int i = tid + u * threads;
      if (i < a.nvec) {
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          w[k] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = (int)fminf(fmaxf(rintf(h[u][4 * k + j] * scale), -127.f), 127.f);
            w[k] |= (uint32_t)(uint8_t)(int8_t)c << (8 * j);
          }
        }
        reinterpret_cast<uint2*>(a.q)[at + i] = uint2{w[0], w[1]};
      }
    }
    if (tid == 0) a.q_scale[row] = top / 127.0f;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <typename T, typename R, typename Wt, int QUANT>
void launch_norm_quant(const NormArgs& a, hipStream_t s) {
  auto go = [&](auto vpt, auto kernel) {
    const int per = decltype(vpt)::value;
    const int threads = ((a.nvec + per - 1) / per + 63) / 64 * 64;
    hipLaunchKernelGGL(kernel, grid_of(a.rows), dim3(threads), 0, s, a);
  };
  // A vector per thread as far as a workgroup has threads: bf16 rows of 7168
  // with y and fp8 out take 184 us (16384 rows) and 3.6 us (32 rows), with two
  // vectors per thread 185 and 4.1, with four 200 and 5.3; rows of 512, 13.0,
  // 13.5 and 14.0 us.  Longer rows need two or four.
  if (a.nvec <= kNormThreads) go(std::integral_constant<int, 1>(), k_add_rms_norm<T, R, Wt, QUANT, 1>);
  else if (a.nvec <= 2 * kNormThreads) go(std::integral_constant<int, 2>(), k_add_rms_norm<T, R, Wt, QUANT, 2>);
  else go(std::integral_constant<int, 4>(), k_add_rms_norm<T, R, Wt, QUANT, 4>);
}

template <typename T, typename R, typename Wt>
void launch_norm(const NormArgs& a, int quant, hipStream_t s) {
  if (quant == MDC_QUANT_INT8) launch_norm_quant<T, R, Wt, MDC_QUANT_INT8>(a, s);
  else if (quant == MDC_QUANT_FP8) launch_norm_quant<T, R, Wt, MDC_QUANT_FP8>(a, s);
  else launch_norm_quant<T, R, Wt, MDC_QUANT_NONE>(a, s);
}

template <typename T>
void launch_norm_typed(const NormArgs& a, const mdc_norm_params& p, hipStream_t s) {
  const bool r32 = p.residual_dtype == MDC_DTYPE_FP32, w32 = p.weight_dtype == MDC_DTYPE_FP32;
  if (r32 && w32) launch_norm<T, float, float>(a, p.quant, s);
  else if (r32) launch_norm<T, float, T>(a, p.quant, s);
  else if (w32) launch_norm<T, T, float>(a, p.quant, s);
  else launch_norm<T, T, T>(a, p.quant, s);
}

}  // namespace

extern "C" {

mdc_status mdc_add_rms_norm(const mdc_norm_params* params, const void* x, const void* residual, const void* weight,
                            void* residual_out, void* y, void* q, float* q_scale, void* stream) {
  if (params == nullptr) return MDC_ERR_NULLPTR;
  const mdc_norm_params& p = *params;
  if (p.dtype != MDC_DTYPE_BF16 && p.dtype != MDC_DTYPE_FP16) return MDC_ERR_INVALID;
  if (p.residual_dtype != p.dtype && p.residual_dtype != MDC_DTYPE_FP32) return MDC_ERR_INVALID;
  if (p.weight_dtype != p.dtype && p.weight_dtype != MDC_DTYPE_FP32) return MDC_ERR_INVALID;
  if (p.quant < MDC_QUANT_NONE || p.quant > MDC_QUANT_FP8) return MDC_ERR_INVALID;
  if (p.rows < 0 || p.hidden <= 0 || p.hidden % 8 != 0) return MDC_ERR_INVALID;
  if (!(p.eps >= 0.f) || !(p.eps - p.eps == 0.f)) return MDC_ERR_INVALID;
  if (p.rows > INT32_MAX || p.hidden > MDC_MAX_NORM_HIDDEN) return MDC_ERR_UNSUPPORTED;
  if (p.rows == 0) return MDC_OK;
  if (x == nullptr || weight == nullptr) return MDC_ERR_NULLPTR;
  if ((p.quant != MDC_QUANT_NONE) != (q != nullptr) || (q != nullptr) != (q_scale != nullptr)) return MDC_ERR_NULLPTR;
  if (residual_out == nullptr && y == nullptr && q == nullptr) return MDC_ERR_NULLPTR;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) || !aligned16(y) ||
      !aligned8(q) || !aligned4(q_scale))
    return MDC_ERR_INVALID;
  const NormArgs a{x,       residual, weight,           residual_out, y, q, q_scale, (int)p.rows, p.hidden / 8,
                   p.eps, 1.0f / (float)p.hidden};
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.dtype == MDC_DTYPE_BF16) launch_norm_typed<Bf16>(a, p, s);
  else launch_norm_typed<_Float16>(a, p, s);
  return launched();
}

}  // extern "C"
