// libmdc: residual addition and RMS norm with 16-bit and 8-bit outputs for
// AMD Instinct MI355X (gfx950): mdc_add_rms_norm.

#include "mdc_rows.h"

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

template <typename T, typename R, typename Wt, int QUANT, int VPT>
__global__ __launch_bounds__(kNormThreads) void k_add_rms_norm(NormArgs a) {
  __shared__ float part[kNormThreads / 64];
  __shared__ uint32_t part_max[kNormThreads / 64];
  const int tid = threadIdx.x, threads = blockDim.x;
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
  const float inv = 1.0f / sqrtf(row_sum(sum, part) * a.inv_hidden + a.eps);
  const NormOut out{a.y, a.q, a.q_scale, a.nvec};
  norm_outputs<T, QUANT, VPT>(out, row, h, inv, part_max, [&](int u, int i, float (&w)[8]) {
    if (a.res_out != nullptr) store8(static_cast<R*>(a.res_out) + (at + i) * 8, h[u]);
    load8(static_cast<const Wt*>(a.weight) + i * 8, w);
  });
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
