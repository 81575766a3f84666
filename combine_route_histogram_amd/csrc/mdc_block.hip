// libmdc: the norms before and after a block with its gate and residual scale,
// for AMD Instinct MI355X (gfx950): mdc_block_rms_norm.

#include "mdc_rows.h"

namespace {

// ---------------------------------------------------------------------------
// h = residual_scale * residual + block_scale * act(gate) * x * inv_x * post,
// with inv_x = 1 / sqrt(mean(x^2) + post_eps) known only after the row was read.
// Everything a row needs is loaded before the sum of x^2: p = x * post * gate and
// the scaled residual stay in registers, and one FMA with inv_x makes h of them.
// (Where both norms are inside fp32's range, p is: it is h's part divided by inv_x.
// With no norm of h, h alone may be larger than that leaves room for.)
// Then h^2 is summed and the outputs leave as for mdc_add_rms_norm.
//
// Sums and everything up to the outputs are fp32; residual_out, y and q are
// rounded once each, from the unrounded values.
//
// Bound: memory.  16384 rows of 7168 (bf16, residual in and out, y, fp8 rows and
// scales: 1.06 GB) 196-203 us, 5.2-5.4 TB/s, where mdc_add_rms_norm takes 184 and a plain
// read and write of its bytes 172: a row waits at one sum more.  With a gate value
// for each element 226 us (5.7 TB/s), with its sigmoid 241: two exact functions of
// fp32, an exponential and a quotient.
// ---------------------------------------------------------------------------
struct BlockArgs {
  const void* x;
  const void* post;      // or NULL: no norm of x
  const void* gate;      // or NULL
  const void* res;       // or NULL
  const void* weight;    // or NULL: residual_out is the only output
  void* res_out;         // or NULL
  NormOut out;
  int rows, nvec;        // vectors of 8 elements per row
  int gate_every;        // rows that share a gate row
  int gate_wide;         // a gate row has a value for each column
  int gate32;            // the gate is fp32
  int act;
  float block_scale, res_scale, post_eps, eps, inv_hidden;
};

// act(g) * scale of n gate values
template <int n>
__device__ __forceinline__ void block_act(float (&g)[n], int act, float scale) {
  if (act == MDC_ACT_SIGMOID) {
#pragma unroll
    for (int j = 0; j < n; ++j) g[j] = 1.0f / (1.0f + expf(-g[j]));
  } else if (act == MDC_ACT_TANH) {
#pragma unroll
    for (int j = 0; j < n; ++j) g[j] = tanhf(g[j]);
  }
#pragma unroll
  for (int j = 0; j < n; ++j) g[j] *= scale;
}

__device__ __forceinline__ float load1(const Bf16* p) { return __uint_as_float((uint32_t)p->bits << 16); }
__device__ __forceinline__ float load1(const _Float16* p) { return (float)*p; }

// Eight elements as they lie in memory, to be loaded now and looked at later.
template <typename T>
struct Raw {
  v4u v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const v4u*>(p); }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    const v4u w = v;
    load8(reinterpret_cast<const T*>(&w), f);
  }
};
template <>
struct Raw<float> {
  v4f a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const v4f*>(p)[0];
    b = reinterpret_cast<const v4f*>(p)[1];
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  }
};

template <typename T, typename R, typename Wt, int QUANT, int VPT>
__global__ __launch_bounds__(kNormThreads) void k_block_rms_norm(BlockArgs a) {
  __shared__ float part[2][kNormThreads / 64];
  __shared__ uint32_t part_max[kNormThreads / 64];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int64_t row = grid_block();
  if (row >= a.rows) return;
  const int64_t at = row * a.nvec;   // first vector of the row
  const int64_t gate_row = (int)row / a.gate_every;
  Raw<T> x[VPT];
  Raw<R> res[VPT];
  Raw<Wt> post[VPT], weight[VPT];
  v4u gate[VPT][2];
  // every load before the first use: one trip to memory for all of them
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = min(tid + u * threads, a.nvec - 1);   // (threads past the row's end load its last vector)
    x[u].load(static_cast<const T*>(a.x) + (at + i) * 8);
    if (a.res != nullptr) res[u].load(static_cast<const R*>(a.res) + (at + i) * 8);
    if (a.gate_wide) {
      const int64_t g = gate_row * a.nvec + i;
      gate[u][0] = static_cast<const v4u*>(a.gate)[a.gate32 ? 2 * g : g];
      if (a.gate32) gate[u][1] = static_cast<const v4u*>(a.gate)[2 * g + 1];
    }
    if (a.post != nullptr) post[u].load(static_cast<const Wt*>(a.post) + i * 8);
    if (VPT < 4 && a.weight != nullptr) weight[u].load(static_cast<const Wt*>(a.weight) + i * 8);
  }
  float gate1[1] = {1.f};
  if (a.gate != nullptr && !a.gate_wide) {
    gate1[0] = a.gate32 ? static_cast<const float*>(a.gate)[gate_row] : load1(static_cast<const T*>(a.gate) + gate_row);
    block_act(gate1, a.act, a.block_scale);
  } else {
    gate1[0] = a.block_scale;
  }
  float h[VPT][8], r[VPT][8];
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const bool in = tid + u * threads < a.nvec;
    x[u].values(h[u]);
    float w[8];
    if (a.post != nullptr) {
      if (in)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[u][j], h[u][j], sum);
      post[u].values(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] *= w[j];
    }
    if (a.gate_wide) {
      if (a.gate32) Raw<float>{__builtin_bit_cast(v4f, gate[u][0]), __builtin_bit_cast(v4f, gate[u][1])}.values(w);
      else Raw<T>{gate[u][0]}.values(w);
      block_act(w, a.act, a.block_scale);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] *= w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] *= gate1[0];
    }
    if (a.res != nullptr) {
      res[u].values(r[u]);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[u][j] *= a.res_scale;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[u][j] = 0.f;
    }
    if (!in)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = r[u][j] = 0.f;
  }
  float inv = 1.f;
  if (a.post != nullptr) inv = 1.0f / sqrtf(row_sum(sum, part[0]) * a.inv_hidden + a.post_eps);
  sum = 0.f;
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = tid + u * threads;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[u][j] = __builtin_fmaf(h[u][j], inv, r[u][j]);
    if (i < a.nvec) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(h[u][j], h[u][j], sum);
      if (a.res_out != nullptr) store8(static_cast<R*>(a.res_out) + (at + i) * 8, h[u]);
    }
  }
  if (a.weight == nullptr) return;
  inv = 1.0f / sqrtf(row_sum(sum, part[1]) * a.inv_hidden + a.eps);
  norm_outputs<T, QUANT, VPT>(a.out, row, h, inv, part_max, [&](int u, int i, float (&w)[8]) {
    if (VPT < 4) weight[u].values(w);
    else load8(static_cast<const Wt*>(a.weight) + i * 8, w);
  });
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <typename T, typename R, typename Wt, int QUANT>
void launch_block_quant(const BlockArgs& a, hipStream_t s) {
  auto go = [&](auto vpt, auto kernel) {
    const int per = decltype(vpt)::value;
    const int threads = ((a.nvec + per - 1) / per + 63) / 64 * 64;
    hipLaunchKernelGGL(kernel, grid_of(a.rows), dim3(threads), 0, s, a);
  };
  // Two vectors a thread from 257 on: smaller workgroups, of which a CU holds more,
  // so that one's waits at its sums are another's loads.  With one, two and four, in
  // us: 16384 rows of 7168 (bf16, a gate row for 2048 rows, y and fp8 out) 238, 202 and
  // 204; 2048 x 7168 with one gate row 36, 33 and 33, 256 rows 7.4, 7.5 and 9.2, 32
  // rows 5.6, 5.6 and 7.1; 2051 x 5000 27.5, 26.0 and 27.8, its int8 rows alone 25.8,
  // 22.2 and 23.6; fp16 with residual and weights in fp32, a sigmoid gate for each
  // element, int8 out 38.1, 38.2 and 39.1; 1000 x 2048 6.9, 7.3 and 9.1; 8192 rows of
  // 16384 234 with two, 242 with four.
  if (a.nvec <= kNormThreads / 4) go(std::integral_constant<int, 1>(), k_block_rms_norm<T, R, Wt, QUANT, 1>);
  else if (a.nvec <= 2 * kNormThreads) go(std::integral_constant<int, 2>(), k_block_rms_norm<T, R, Wt, QUANT, 2>);
  else go(std::integral_constant<int, 4>(), k_block_rms_norm<T, R, Wt, QUANT, 4>);
}

template <typename T, typename R, typename Wt>
void launch_block(const BlockArgs& a, int quant, hipStream_t s) {
  if (quant == MDC_QUANT_INT8) launch_block_quant<T, R, Wt, MDC_QUANT_INT8>(a, s);
  else if (quant == MDC_QUANT_FP8) launch_block_quant<T, R, Wt, MDC_QUANT_FP8>(a, s);
  else launch_block_quant<T, R, Wt, MDC_QUANT_NONE>(a, s);
}

template <typename T>
void launch_block_typed(const BlockArgs& a, const mdc_block_norm_params& p, hipStream_t s) {
  const bool r32 = p.residual_dtype == MDC_DTYPE_FP32, w32 = p.weight_dtype == MDC_DTYPE_FP32;
  if (r32 && w32) launch_block<T, float, float>(a, p.quant, s);
  else if (r32) launch_block<T, float, T>(a, p.quant, s);
  else if (w32) launch_block<T, T, float>(a, p.quant, s);
  else launch_block<T, T, T>(a, p.quant, s);
}

bool finite(float v) { return v - v == 0.f; }

}  // namespace

extern "C" {

mdc_status mdc_block_rms_norm(const mdc_block_norm_params* params, const void* x, const void* post_weight,
                              const void* gate, const void* residual, const void* weight, void* residual_out, void* y,
                              void* q, float* q_scale, void* stream) {
  if (params == nullptr) return MDC_ERR_NULLPTR;
  const mdc_block_norm_params& p = *params;
  if (p.dtype != MDC_DTYPE_BF16 && p.dtype != MDC_DTYPE_FP16) return MDC_ERR_INVALID;
  for (int32_t t : {p.residual_dtype, p.weight_dtype, p.gate_dtype})
    if (t != p.dtype && t != MDC_DTYPE_FP32) return MDC_ERR_INVALID;
  if (p.quant < MDC_QUANT_NONE || p.quant > MDC_QUANT_FP8) return MDC_ERR_INVALID;
  if (p.gate_act < MDC_ACT_NONE || p.gate_act > MDC_ACT_TANH) return MDC_ERR_INVALID;
  if (p.rows < 0 || p.hidden <= 0 || p.hidden % 8 != 0) return MDC_ERR_INVALID;
  if (p.gate_columns != 1 && p.gate_columns != p.hidden) return MDC_ERR_INVALID;
  if (p.gate_every < 1) return MDC_ERR_INVALID;
  if (!(p.eps >= 0.f) || !finite(p.eps) || !(p.post_eps >= 0.f) || !finite(p.post_eps)) return MDC_ERR_INVALID;
  if (!finite(p.block_scale) || !finite(p.residual_scale)) return MDC_ERR_INVALID;
  if (p.rows > INT32_MAX || p.hidden > MDC_MAX_NORM_HIDDEN) return MDC_ERR_UNSUPPORTED;
  if (p.rows == 0) return MDC_OK;
  if (x == nullptr) return MDC_ERR_NULLPTR;
  if ((p.quant != MDC_QUANT_NONE) != (q != nullptr) || (q != nullptr) != (q_scale != nullptr)) return MDC_ERR_NULLPTR;
  if (residual_out == nullptr && y == nullptr && q == nullptr) return MDC_ERR_NULLPTR;
  if (weight == nullptr && (y != nullptr || q != nullptr)) return MDC_ERR_NULLPTR;
  const bool wide = gate != nullptr && p.gate_columns != 1;
  if (!aligned16(x) || !aligned16(post_weight) || !aligned16(residual) || !aligned16(weight) ||
      !aligned16(residual_out) || !aligned16(y) || !aligned8(q) || !aligned4(q_scale))
    return MDC_ERR_INVALID;
  const uintptr_t unit = wide ? 16 : p.gate_dtype == MDC_DTYPE_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(gate) % unit != 0) return MDC_ERR_INVALID;
  const int nvec = p.hidden / 8;
  if (y == nullptr && q == nullptr) weight = nullptr;   // (nothing to normalise for)
  const BlockArgs a{x, post_weight, gate, residual, weight, residual_out, NormOut{y, q, q_scale, nvec}, (int)p.rows, nvec,
                    (int)(p.gate_every < p.rows ? p.gate_every : p.rows), wide, p.gate_dtype == MDC_DTYPE_FP32, p.gate_act,
                    p.block_scale, p.residual_scale, p.post_eps, p.eps, 1.0f / (float)p.hidden};
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.dtype == MDC_DTYPE_BF16) launch_block_typed<Bf16>(a, p, s);
  else launch_block_typed<_Float16>(a, p, s);
  return launched();
}

}  // extern "C"
