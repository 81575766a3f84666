// libmdc: routing of tokens to experts for AMD Instinct MI355X (gfx950):
// mdc_gate, whose ids and weights are the expert_ids and expert_scales of the
// dispatch and the combine.

#include "mdc_gate.h"

namespace {

template <typename T, int LPT, int VPL>
__global__ __launch_bounds__(kGateThreads) void k_gate(GateArgs a) {
  extern __shared__ int64_t gate_lds[];
  constexpr int kTokens = kGateThreads / LPT;
  const int lane = threadIdx.x & (LPT - 1);
  const int slot = threadIdx.x / LPT;
  const int64_t token = grid_block() * kTokens + slot;
  // (lanes past the last token repeat it and store nothing)
  gate_token<T, LPT, VPL>(a, min(token, (int64_t)a.T - 1), token < a.T, lane,
                          gate_lds + (int64_t)slot * (LPT * VPL + (LPT * VPL >> 5)));
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
  const mdc_status gate = check_gate(p, E, shape->topk);
  if (gate != MDC_OK) return gate;
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
