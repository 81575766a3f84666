// Grouped products: rows and tiles of the experts, worked out from the counts on
// the device, and what their kernels share besides.  A problem is a struct with
// nums (rows of each expert, or NULL: one expert with all rows), A (capacity)
// and L (experts).
#pragma once

#include "mdc_fp8.h"

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(4))) float scalar_f;   // read by scalar loads

// A value that all lanes share, in a scalar register (a choice between two of them
// does not become a vector load of the one chosen).
__device__ __forceinline__ float scalar(float v) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))); }

__device__ __forceinline__ v8i join(v4i a, v4i b) { return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

// By the hardware's exp and reciprocal, about 1 ulp each (the exponential's argument is
// rounded to fp32 before, so that its error grows with |a|): what follows rounds the
// value to 8 bits, and exact functions would cost several times the instructions.
__device__ __forceinline__ float gmm_silu(float a) { return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }

constexpr unsigned kPastEnd = 0x80000000u;   // an offset past every buffer: loads there read zero
__device__ __forceinline__ unsigned lds_at(const void* p) { return (unsigned)(size_t)(lds_void*)p; }
__device__ __forceinline__ void lds_put(unsigned at, v4f v) {
  asm volatile("ds_write_b128 %0, %1" ::"v"(at), "v"(v) : "memory");
}
// Sums of v_mfma_i32_16x16x64_i8 that lds_put writes next: of an instruction in inline
// assembly the compiler does not know that it reads them, and leaves out the 8 wait
// states that the matrix instruction's results take.
template <int n>
__device__ __forceinline__ void matrix_hold(v4i (&acc)[n]) {
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" : "+v"(acc[i]));
}
template <int m, int n>
__device__ __forceinline__ void matrix_hold(v4i (&acc)[m][n]) {
#pragma unroll
  for (int i = 0; i < m; ++i) matrix_hold(acc[i]);
}
template <typename Sums>
__device__ __forceinline__ void matrix_done(Sums& acc) {
  matrix_hold(acc);
  asm volatile("s_nop 7");
}
__device__ __forceinline__ v8i lds_get2(unsigned a, unsigned b) {
  v4i x, y;
  asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x), "=&v"(y)
               : "v"(a), "v"(b)
               : "memory");
  return join(x, y);
}
// a barrier that leaves loads in flight
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---------------------------------------------------------------------------
// Rows and tiles of the experts.  Every workgroup works out the plan from the
// counts by itself, in LDS.  Experts with at most kThinRows rows, two blocks of
// the matrix instruction, are "thin": what counts there is to stream the
// weights.  The others are "wide".
// ---------------------------------------------------------------------------
constexpr int kGmmThreads = 512;
constexpr int kGmmWaves = kGmmThreads / 64;
constexpr int kThinBlocks = 2;
constexpr int kThinRows = 16 * kThinBlocks;

struct GmmTable {
  int* rows;        // [L + 1] first row of expert e
  int* tiles;       // [L + 1] first m-tile of expert e (tiles of wide experts)
  uint16_t* thin;   // [L] the thin experts with rows
  int n_thin;
};
constexpr size_t gmm_table_bytes(int L) { return 2 * sizeof(int) * ((size_t)L + 1) + sizeof(uint16_t) * (size_t)L; }

// Inclusive sum over the workgroup's threads, and the sum of all of them.
// wave_total holds a value per wavefront.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* wave_total, int64_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // in two halves of at most 30 bits' sum each: 0 <= v < 2^48
  const int64_t low = wave_inclusive_scan((int)(v & 0xFFFFFF));
  v = ((int64_t)wave_inclusive_scan((int)(v >> 24)) << 24) + low;
  if (lane == 63) wave_total[wave] = v;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    const int64_t n = wave_total[w];
    if (w < wave) v += n;
    all += n;
  }
  __syncthreads();
  return v;
}

// Rows of expert e as counted (negative: none).
__device__ __forceinline__ int64_t gmm_count(const int64_t* nums, int e, int64_t A) {
  return nums == nullptr ? A : min(max(nums[e], (int64_t)0), A);
}

// rows[e] of every expert, clipped at A.
template <int THREADS, typename G>
__device__ __forceinline__ void gmm_rows(const G& g, int* rows, int64_t* wave_total) {
  int64_t carry = 0, all;
  for (int e0 = 0; e0 < g.L; e0 += THREADS) {
    const int e = e0 + threadIdx.x;
    const int64_t end = carry + block_scan<THREADS>(e < g.L ? gmm_count(g.nums, e, g.A) : 0, wave_total, all);
    if (e < g.L) rows[e + 1] = (int)min(end, (int64_t)g.A);
    carry += all;
  }
  if (threadIdx.x == 0) rows[0] = 0;
  __syncthreads();
}

// The thin experts, and tiles[e] with m-tiles of `rows` rows.  Returns the
// number of m-tiles.
template <typename G>
__device__ __forceinline__ int gmm_tiles(const G& g, GmmTable& t, int rows, int64_t* wave_total) {
  int64_t carry = 0, all;   // m-tiles so far, and thin experts above 2^32
  for (int e0 = 0; e0 < g.L; e0 += kGmmThreads) {
    const int e = e0 + threadIdx.x;
    const int n = e < g.L ? t.rows[e + 1] - t.rows[e] : 0;
    const bool thin = n > 0 && n <= kThinRows;
    const int64_t mine = thin ? (int64_t)1 << 32 : n > 0 ? (n - 1) / rows + 1 : 0;   // (n up to 2^31 - 1)
    const int64_t end = carry + block_scan<kGmmThreads>(mine, wave_total, all);
    if (e < g.L) t.tiles[e + 1] = (int)(uint32_t)end;
    if (thin) t.thin[(int)(end >> 32) - 1] = (uint16_t)e;
    carry += all;
  }
  if (threadIdx.x == 0) t.tiles[0] = 0;
  __syncthreads();
  t.n_thin = __builtin_amdgcn_readfirstlane((int)(carry >> 32));
  return __builtin_amdgcn_readfirstlane((int)(uint32_t)carry);
}

// Numbers of m-tiles of 128, 64 and 32 rows (at most 2^26 + L each).
template <typename G>
__device__ __forceinline__ void gmm_tile_counts(const G& g, const GmmTable& t, int (&count)[3]) {
  int n[3] = {0, 0, 0};
  for (int e = threadIdx.x; e < g.L; e += kGmmThreads) {
    const int rows = t.rows[e + 1] - t.rows[e];
    if (rows > kThinRows)
#pragma unroll
      for (int i = 0; i < 3; ++i) n[i] += (rows - 1) / (128 >> i) + 1;
  }
  __shared__ int part[3][kGmmWaves];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    n[i] = wave_inclusive_scan(n[i]);
    if ((threadIdx.x & 63) == 63) part[i][threadIdx.x >> 6] = n[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    count[i] = 0;
#pragma unroll
    for (int w = 0; w < kGmmWaves; ++w) count[i] += part[i][w];
    count[i] = __builtin_amdgcn_readfirstlane(count[i]);
  }
}

// Expert that m-tile m belongs to: the number of experts whose tiles end at or
// before m.
__device__ __forceinline__ int gmm_expert(const GmmTable& t, int L, int m) {
  const int lane = threadIdx.x & 63;
  int e = 0;
  for (int e0 = 0; e0 < L; e0 += 64) {
    const int i = e0 + lane;
    e += __popcll(__ballot(i < L && t.tiles[i + 1] <= m));
  }
  return __builtin_amdgcn_readfirstlane(e);
}

// This workgroup's place in the walks: workgroup b runs on XCD b % 8, and each
// XCD takes a run of places.
__device__ __forceinline__ int wide_line() { return (blockIdx.x % 8) * (gridDim.x / 8) + blockIdx.x / 8; }

// First of T equal pieces of thin work for the workgroup at place `line`, after
// `wide` wide tiles were dealt to places 0, 1, ... in turn: a place with a wide
// tile more gets less, a wide tile counted as `cost` pieces.
__device__ __forceinline__ int64_t thin_share(int64_t T, int wide, int cost, int line) {
  const int G = gridDim.x, more = wide % G;   // places [0, more) have a tile more
  // x pieces for those, x + cost for the others: more x + (G - more) (x + cost) = T, x >= 0
  const int64_t rest = T - (int64_t)(G - more) * cost;
  if (rest <= 0) return line <= more ? 0 : T * (line - more) / (G - more);   // (more < G)
  return line <= more ? rest * line / G : rest * line / G + (int64_t)(line - more) * cost;
}

struct WideTile {
  int e, row0, rows, n0;   // n0: first weight row (SwiGLU: first output column)
};

// Tile number -> place.  The m-tiles of an expert run in chunks of up to 8,
// and a chunk's tiles in groups of h m-tiles x 32 / h n-tiles, m fastest, so
// that the about 32 tiles an XCD runs at a time share rows and weights in its
// L2.
template <typename G>
__device__ __forceinline__ WideTile wide_place(const G& g, const GmmTable& tab, int t, int nn, int BM, int cols) {
  const int m = t / nn;
  const int e = gmm_expert(tab, g.L, m);
  const int m_first = tab.tiles[e], m_end = tab.tiles[e + 1];
  const int c0 = m_first + (m - m_first) / 8 * 8;
  const int h = min(8, m_end - c0);
  const int r = t - c0 * nn;
  const int gn = 32 / h, band = h * gn;
  const int ng = r / band, r2 = r - ng * band;
  const int q = r2 / h;
  const int mt = c0 + (r2 - q * h);
  WideTile w;
  w.e = e;
  w.row0 = __builtin_amdgcn_readfirstlane(tab.rows[e] + (mt - m_first) * BM);
  w.rows = __builtin_amdgcn_readfirstlane(min(tab.rows[e + 1] - w.row0, BM));
  w.n0 = __builtin_amdgcn_readfirstlane((ng * gn + q) * cols);
  return w;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
unsigned device_cus() {
  int dev = 0, cus = 256;
  if (hipGetDevice(&dev) == hipSuccess) (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  return (unsigned)cus;
}

constexpr size_t kLdsSize = 160 << 10;   // of a CU

}  // namespace
