// libmdc: grouped product in int8 with a scale for each row and each output
// channel, for AMD Instinct MI355X (gfx950): mdc_gmm_int8.

#include "mdc_group.h"

namespace {

// ---------------------------------------------------------------------------
// y[r][c] = (sum over k of a[r][k] w[e][c][k]) * sa[r] * sw[e][c].  The sum is
// exact (int32: K < 2^17), the factors are applied once at the end, in this
// order, each product rounded to fp32.
//
// The weight block is the first operand of the matrix instruction and the token
// block the second, so that a lane ends up with runs of four consecutive output
// columns of one token.
// ---------------------------------------------------------------------------
typedef int v16i __attribute__((ext_vector_type(16)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));

struct Gmm8 {
  const int8_t* a;         // [A][K]
  const float* a_scale;    // [A]
  const int64_t* nums;     // [L], or NULL: one expert with all A rows
  const int8_t* w;         // [L][Nw][K]
  const float* w_scale;    // [L][Nw]
  void* y;                 // [A][Nw]
  int A, L, Nw, K, nk;     // nk: k-blocks of 128
  int dtype;               // of y
};

constexpr int kGmm8Block = 128;          // bytes of k of a stage

// Four output columns of one row.
__device__ __forceinline__ v4f gmm8_scale(v4i acc, float sa, v4f sw) {
  v4f v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = (float)acc[r] * sa * sw[r];
  return v;
}
__device__ __forceinline__ void gmm8_store(const Gmm8& g, int64_t at, v4f v) {
  if (g.dtype == MDC_DTYPE_FP32) *reinterpret_cast<v4f*>(static_cast<float*>(g.y) + at) = v;
  else if (g.dtype == MDC_DTYPE_BF16) *reinterpret_cast<v4b*>(static_cast<uint16_t*>(g.y) + at) = __builtin_convertvector(v, v4b);
  else *reinterpret_cast<v4h*>(static_cast<uint16_t*>(g.y) + at) = __builtin_convertvector(v, v4h);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t channel_scales(const Gmm8& g, int e) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(g.w_scale + (int64_t)e * g.Nw), (short)0, g.Nw * 4, 0x00020000);
}

// ---------------------------------------------------------------------------
// Tiles of 64 rows x 64 columns, four wavefronts of 32 x 32 each; k in stages of
// 128 bytes through LDS.  Chunk c (16 bytes) of row r sits at chunk c ^ ((r / 2) &
// 7) of the row's 128 bytes, so that the reads of a fragment cover all banks.
// ---------------------------------------------------------------------------
constexpr int kSimple = 64;

__global__ __launch_bounds__(kGmmThreads) void k_gmm8(Gmm8 g) {
  extern __shared__ int gmm_table[];
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * kSimple * kGmm8Block];
  __shared__ int64_t wave_total[kGmmWaves];
  GmmTable tab{gmm_table, gmm_table + g.L + 1, reinterpret_cast<uint16_t*>(gmm_table + 2 * (g.L + 1)), 0};
  gmm_rows<kGmmThreads>(g, tab.rows, wave_total);
  // every expert as a wide one
  int64_t carry = 0, all;
  for (int e0 = 0; e0 < g.L; e0 += kGmmThreads) {
    const int e = e0 + threadIdx.x;
    const int n = e < g.L ? tab.rows[e + 1] - tab.rows[e] : 0;
    const int64_t end = carry + block_scan<kGmmThreads>(n > 0 ? (n - 1) / kSimple + 1 : 0, wave_total, all);
    if (e < g.L) tab.tiles[e + 1] = (int)end;
    carry += all;
  }
  if (threadIdx.x == 0) tab.tiles[0] = 0;
  __syncthreads();
  const int nn = (g.Nw + kSimple - 1) / kSimple;
  const int T = tab.tiles[g.L] * nn;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wt = (wave >> 1) & 1, wn = wave & 1;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const int m = t / nn, n0 = (t - m * nn) * kSimple;
    const int e = gmm_expert(tab, g.L, m);
    const int row0 = tab.rows[e] + (m - tab.tiles[e]) * kSimple, rows = min(kSimple, tab.rows[e + 1] - row0);
    v16i acc = v16i{};
    for (int b = 0; b < g.nk; ++b) {
      __syncthreads();
      // thread (row, chunk) of 128 rows (tokens, then weights): two chunks each
      for (int i = tid; i < 2 * kSimple * 8; i += kGmmThreads) {
        const int r = i >> 3, c = i & 7, k = b * kGmm8Block + 16 * c;
        v4i v = {0, 0, 0, 0};
        if (k < g.K) {
          if (r < kSimple) {
            if (r < rows) v = *reinterpret_cast<const v4i*>(g.a + (int64_t)(row0 + r) * g.K + k);
          } else if (n0 + r - kSimple < g.Nw) {
            v = *reinterpret_cast<const v4i*>(g.w + ((int64_t)e * g.Nw + n0 + r - kSimple) * g.K + k);
          }
        }
        *reinterpret_cast<v4i*>(smem + r * kGmm8Block + ((c ^ ((r >> 1) & 7)) << 4)) = v;
      }
      __syncthreads();
      if (wave < 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int rt = 32 * wt + (lane & 31), rw = kSimple + 32 * wn + (lane & 31), c = 2 * q + (lane >> 5);
          const v4i ft = *reinterpret_cast<const v4i*>(smem + rt * kGmm8Block + ((c ^ ((rt >> 1) & 7)) << 4));
          const v4i fw = *reinterpret_cast<const v4i*>(smem + rw * kGmm8Block + ((c ^ ((rw >> 1) & 7)) << 4));
          acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw, ft, acc, 0, 0, 0);
        }
      }
    }
    const int r = 32 * wt + (lane & 31);
    if (wave < 4 && r < rows) {
      const __amdgpu_buffer_rsrc_t rc = channel_scales(g, e);
      const float sa = g.a_scale[row0 + r];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = n0 + 32 * wn + 8 * q + 4 * (lane >> 5);
        if (col < g.Nw) {
          const v4f sw = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rc, col * 4, 0, 0));
          gmm8_store(g, (int64_t)(row0 + r) * g.Nw + col, gmm8_scale(v4i{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]}, sa, sw));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
void launch_gmm8(const Gmm8& g, hipStream_t s) {
  const dim3 grid((device_cus() + 7) / 8 * 8), block(kGmmThreads);
  hipLaunchKernelGGL(k_gmm8, grid, block, gmm_table_bytes(g.L), s, g);
}

constexpr int kGmm8MaxK = 1 << 17;   // below it 2^14 K fits 32 bits

mdc_status check_gmm8(int64_t A, int32_t L, int32_t n, int32_t k) {
  if (A < 0 || L < 1 || n < 1 || k < 1 || n % 8 != 0 || k % 16 != 0) return MDC_ERR_INVALID;
  if (L > MDC_MAX_LOCAL_EXPERTS || A > INT32_MAX || (int64_t)n * k > INT32_MAX || k >= kGmm8MaxK) return MDC_ERR_UNSUPPORTED;
  if ((A / kThinRows + L + 1) * ((n + 15) / 16) > INT32_MAX - 65536) return MDC_ERR_UNSUPPORTED;
  return MDC_OK;
}

}  // namespace

extern "C" {

mdc_status mdc_gmm_int8(int64_t capacity, int32_t experts, int32_t n, int32_t k, int32_t y_dtype, const int8_t* a,
                        const float* a_scale, const int64_t* expert_token_nums, const int8_t* w, const float* w_scale,
                        void* y, void* stream) {
  if (y_dtype < MDC_DTYPE_BF16 || y_dtype > MDC_DTYPE_FP32) return MDC_ERR_INVALID;
  const mdc_status st = check_gmm8(capacity, experts, n, k);
  if (st != MDC_OK) return st;
  if (capacity == 0) return MDC_OK;
  if (a == nullptr || a_scale == nullptr || w == nullptr || w_scale == nullptr || y == nullptr ||
      (expert_token_nums == nullptr && experts != 1))
    return MDC_ERR_NULLPTR;
  if (!aligned16(a) || !aligned4(a_scale) || !aligned8(expert_token_nums) || !aligned16(w) || !aligned4(w_scale) ||
      !aligned16(y))
    return MDC_ERR_INVALID;
  (void)hipGetLastError();
  launch_gmm8(Gmm8{a, a_scale, expert_token_nums, w, w_scale, y, (int)capacity, experts, n, k,
                   (k + kGmm8Block - 1) / kGmm8Block, y_dtype},
              static_cast<hipStream_t>(stream));
  return launched();
}

}  // extern "C"
