// Rows in registers, a workgroup for each: what the norms share.  Thread t holds
// the row's vectors t, t + threads, ... of 8 elements.
#pragma once

#include "mdc_fp8.h"

namespace {

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

// Sum over the workgroup's threads; part holds a value per wavefront.
__device__ __forceinline__ float row_sum(float v, float* part) {
  const int tid = threadIdx.x, waves = blockDim.x >> 6;
  v = wave_sum(v);
  if ((tid & 63) == 0) part[tid >> 6] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < waves; ++w) v += part[w];
  return v;
}

struct NormOut {
  void* y;          // or NULL
  void* q;          // or NULL
  float* q_scale;
  int nvec;         // vectors of 8 elements per row
};

// Outputs of a row: v = h * inv * weight rounded to T, and in 8 bits.  weight(u,
// i, w) gives the eight weights of the thread's vector u, which is vector i of
// the row; part_max holds a value per wavefront.
template <typename T, int QUANT, int VPT, typename F>
__device__ __forceinline__ void norm_outputs(const NormOut& o, int64_t row, float (&h)[VPT][8], float inv,
                                             uint32_t* part_max, F&& weight) {
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
  const int64_t at = row * o.nvec;   // first vector of the row
  uint32_t amax = 0;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = tid + u * threads;
    float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // h * weight, v before the row's factor
    if (i < o.nvec) {
      float w[8];
      weight(u, i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (QUANT == MDC_QUANT_FP8) t[j] = h[u][j] * w[j];
        h[u][j] = h[u][j] * inv * w[j];   // (h times a large or tiny weight may leave fp32)
      }
      if (o.y != nullptr) store8(static_cast<T*>(o.y) + (at + i) * 8, h[u]);
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
      if (i < o.nvec) {
        reinterpret_cast<uint2*>(o.q)[at + i] = uint2{s.codes4(t[0], t[1], t[2], t[3]),
                                                      s.codes4(t[4], t[5], t[6], t[7])};
        if ((i & 15) == 0) o.q_scale[row * ((o.nvec + 15) >> 4) + (i >> 4)] = s.scale;
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
      if (i < o.nvec) {
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
        reinterpret_cast<uint2*>(o.q)[at + i] = uint2{w[0], w[1]};
      }
    }
    if (tid == 0) o.q_scale[row] = top / 127.0f;
  }
}

}  // namespace
