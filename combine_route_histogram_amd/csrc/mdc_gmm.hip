// libmdc: grouped products in fp8 (e4m3) with a scale for each block of 128,
// and the expert FFN built on them, for AMD Instinct MI355X (gfx950):
// mdc_gmm_fp8, mdc_ffn_fp8, mdc_ffn_fp8_quant_input.

#include "mdc_fp8.h"

namespace {

// ---------------------------------------------------------------------------
// y[r][c] = sum over k-blocks b of sa[r][b] sw[e][c / 128][b] P_b[r][c], where
// P_b is the plain product over 128 columns.  v_mfma_f32_16x16x128_f8f6f4
// multiplies exactly one such block: each instruction starts from zero, and
// its 16 x 16 result is added to the fp32 accumulators with the block's scale
// by four FMAs per lane, which run beside the next matrix instructions.
//
// The weight block is the first operand and the token block the second: lane l
// supplies row l % 16 of each and receives C[4 (l / 16) + i][l % 16], i < 4,
// i.e. four consecutive output columns of one token, so that one scale per
// lane serves a 16 x 16 block.  The 32 bytes a lane supplies are the 16-byte
// chunks l / 16 and 4 + l / 16 of its row's 128: which k they are does not
// matter, as long as both operands agree.
//
// Inside an instruction the products of eight consecutive k are cut to a
// multiple of 2^(E - 13), E the sum of the exponents of the largest product's
// factors, and added exactly; the sums of eights are added in fp32.  Products of
// two e4m3 significands have 8 bits, so only those far below the largest lose
// any.  Nothing else is below fp32 until y is rounded to bf16 (or g to e4m3).
//
// Bounds (bf16 out).  Few rows per expert: memory, 256 rows of 30 experts x 4096
// x 7168 (883 MB of weights) 168 us, 5.27 TB/s, where a plain read of 1 GiB reaches
// 7.1.  Many rows: the matrix units have work for 38 to 47% of the time, at 1.9 to
// 2.1 GHz in place of 2.4; 2048 x 4096 x 7168 on one expert 60 us, 2.0 PFLOP/s, as
// fast as the library's product with one scale for all; 16384 rows of 16 experts,
// both products of an FFN, 752 us, 1.9 PFLOP/s, where the library's keeps the units
// busy for 76% of the time at the same clock (2.6 PFLOP/s): the direct loads are a
// quarter of a stage and the scales' FMAs a seventh.  Up to a few hundred rows on
// few experts: the number of k-blocks one workgroup walks, one after another
// (48 rows of one expert x 4096 x 7168 take 45 us and 256 rows 46, on 32 of the 256
// CUs and on 128; 512 rows, both products, 49 us).
// ---------------------------------------------------------------------------
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(4))) float scalar_f;   // read by scalar loads

__device__ __forceinline__ v4f mfma_block(v8i w, v8i t) {
  // formats 0, 0: both operands e4m3; no hardware scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, t, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v8i join(v4i a, v4i b) { return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

__device__ __forceinline__ float gmm_silu(float a) { return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }

// One grouped product.
struct Gmm {
  const uint8_t* a;        // [A][K] e4m3
  const float* a_scale;    // [A][nk]
  const int64_t* nums;     // [L], or NULL: one expert with all A rows
  const uint8_t* w;        // [L][Nw][K] e4m3
  const float* w_scale;    // [L][ceil(Nw / 128)][nk]
  uint16_t* y;             // [A][Nw] bf16
  float* g;                // SwiGLU with split: [A][Nw / 2] fp32
  uint8_t* q;              // SwiGLU: [A][Nw / 2] e4m3
  float* q_scale;          // [A][Nw / 256]
  mdc_device_status* status;   // cleared, or NULL
  int A, L, Nw, K, nk;
  int split;               // SwiGLU: thin experts' outputs go through g
};

// ---------------------------------------------------------------------------
// Rows and tiles of the experts.  Every workgroup works out the plan from the
// counts by itself, in LDS.  Experts with at most kThinRows rows, two blocks of
// the matrix instruction, are "thin": what counts there is to stream the
// weights.  The others are "wide".  Where the border lies between 16 and 32 rows
// makes no difference to the 256 rows above, 1 to 32 of them an expert (167 and 168
// us).  24 rows an expert x 4096 x 7168, thin : wide, in us: 1 expert 19 : 47, 4
// experts 35 : 55, 8 experts 58 : 65, 16 experts 101 : 88, 32 experts 193 : 166.
// The border is at 32 for the few experts' sake, where the wide tiles leave most
// CUs idle; many experts with 17 to 32 rows each pay up to 20% for it.
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
template <int THREADS>
__device__ __forceinline__ void gmm_rows(const Gmm& g, int* rows, int64_t* wave_total) {
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
__device__ __forceinline__ int gmm_tiles(const Gmm& g, GmmTable& t, int rows, int64_t* wave_total) {
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
__device__ __forceinline__ void gmm_tile_counts(const Gmm& g, const GmmTable& t, int (&count)[3]) {
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

// ---------------------------------------------------------------------------
// Thin experts.  A tile is one expert's rows times 16 rs output columns (SwiGLU:
// of gate and of up): wavefront (rb, kh) takes 16 weight rows of it over the
// kh-th of ks runs of k-blocks, rs ks = 8, and the runs' sums are joined through
// LDS.  A workgroup takes a run of consecutive tiles.
//
// The weights, which are all that memory has to bring, go global -> LDS
// directly, eight rows x 128 bytes per instruction, into a ring of each
// wavefront's own, kThinRing bytes ahead and on into the next tile.  (Loads in
// the matrix instruction's layout, 16 rows x 64 bytes, cost the address unit 27
// ns per KB instead of 7 and kept a decode step's weights at 4.0 TB/s.)  The
// expert's rows stay in registers from tile to tile, kThinRun k-blocks of them.
//
// The compiler would make every LDS access wait for every direct load in
// flight, so the accesses here are written out with their waits: a ring slot is
// read when at most the loads of the slots behind it are out.  Other memory
// operations in between only make that wait longer.
//
// SwiGLU's outputs are quantised in blocks of 128 columns: a workgroup takes
// whole blocks and collects them in LDS (Gmm.split: it takes tiles, and their
// outputs go to memory in fp32, where k_quant_fp8_thin quantises them).
// ---------------------------------------------------------------------------
constexpr unsigned kPastEnd = 0x80000000u;   // an offset past every buffer: loads there read zero
constexpr int kThinRing = 12288;             // bytes of a wavefront's ring
constexpr int kThinRun = 8;                  // k-blocks of rows in registers
constexpr int kWideCost = 2;                 // a wide tile's time in those of 128 columns of thin work
constexpr int kLineG = kFp8Block + 4;        // floats of a row of SwiGLU outputs in LDS

__device__ __forceinline__ unsigned lds_at(const void* p) { return (unsigned)(size_t)(lds_void*)p; }
__device__ __forceinline__ void lds_put(unsigned at, v4f v) {
  asm volatile("ds_write_b128 %0, %1" ::"v"(at), "v"(v) : "memory");
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

struct ThinSmem {
  unsigned ring;   // this wavefront's, kThinRing bytes
  unsigned red;    // [8 wavefronts][1 or 2 blocks][64] v4f
  unsigned g;      // [kThinRows][kLineG] fp32
};

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

template <bool GLU>
__device__ __forceinline__ void thin_walk(const Gmm& g, const GmmTable& tab, int wide, int ks, const ThinSmem& sm) {
  constexpr int WB = GLU ? 2 : 1, MB = kThinBlocks;
  constexpr int kSlot = WB * 2048, kSlots = kThinRing / kSlot;
  constexpr int kLoads = 2 * WB;   // direct loads of a slot
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const int K = g.K, nk = g.nk, Nw = g.Nw, cols = GLU ? Nw / 2 : Nw;
  const int wb = (Nw + kFp8Block - 1) / kFp8Block;
  const int rs = kGmmWaves / ks, rb = wave / ks, kh = wave - rb * ks;
  const int per = (nk + ks - 1) / ks, kb0 = kh * per;
  const bool blocks = GLU && !g.split;               // whole 128-column blocks per workgroup
  const int width = 16 * rs, tiles_per = (cols + width - 1) / width;
  // this workgroup's tiles: [t0, t1) of n_thin * tiles_per, whole blocks of ks tiles if they are wanted
  const int grain = blocks ? ks : 1;
  const int64_t T = (int64_t)tab.n_thin * tiles_per / grain;
  const int cost = max(1, kWideCost * 8 / (rs * grain));
  const int t0 = (int)thin_share(T, wide, cost, wide_line()) * grain;
  const int t1 = (int)thin_share(T, wide, cost, wide_line() + 1) * grain;
  if (t0 == t1) return;

  // ---- weights: tile by tile, step by step ----
  auto weights = [&](int i) {
    const int e = __builtin_amdgcn_readfirstlane((int)tab.thin[i]);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.w + (int64_t)e * Nw * K), (short)0, Nw * K,
                                             0x00020000);
  };
  struct {
    int i, n, step, left;   // place of the expert in the list, first column, step, tiles to come
  } c = {t0 / tiles_per, (t0 % tiles_per) * width, 0, t1 - t0};
  __amdgpu_buffer_rsrc_t rw = weights(c.i);
  unsigned slot = 0;   // of the next load
  const int lrow = lane >> 3;
  auto fetch = [&]() {
    const bool in = c.left > 0;
    const unsigned k0 = in ? (unsigned)min(kb0 + c.step, nk) * kFp8Block : (unsigned)nk * kFp8Block;
#pragma unroll
    for (int j = 0; j < WB; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {   // rows 8 h + lane / 8; the chunk whose place lane % 8 is
        const unsigned chunk = (unsigned)((lane & 7) ^ ((4 * h + (lrow >> 1)) & 7)) << 4;
        const int row = c.n + 16 * rb + 8 * h + lrow;
        const bool ok = k0 + chunk < (unsigned)K && row < cols;
        const unsigned at = ok ? (unsigned)(row + j * (Nw / 2)) * (unsigned)K + k0 + chunk : kPastEnd;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(size_t)(sm.ring + slot + j * 2048 + h * 1024), 16, at,
                                                 0, 0, 0);
      }
    }
    slot = slot + kSlot == kSlots * kSlot ? 0 : slot + kSlot;
    if (++c.step == per) {
      c.step = 0;
      --c.left;
      c.n += width;
      if (c.n >= cols) {
        c.n = 0;
        if (c.left > 0) rw = weights(++c.i);
      }
    }
  };
#pragma unroll
  for (int d = 0; d < kSlots; ++d) fetch();

  const int key = (r16 >> 1) & 7;
  const unsigned f0 = sm.ring + r16 * kFp8Block + ((quad ^ key) << 4);
  const unsigned f1 = sm.ring + r16 * kFp8Block + (((4 + quad) ^ key) << 4);
  unsigned read = 0;
  v8i tok[kThinRun][MB];
  float sa[kThinRun][MB], sw[WB][kThinRun], sw_next[WB][kThinRun];
  // weight scales of a tile's run, by scalar loads: they pass by the direct loads' count
  auto scales = [&](float (&s)[WB][kThinRun], int e, int n, int s0) {
    const scalar_f* p = (const scalar_f*)(g.w_scale + ((int64_t)e * wb + min((n + 16 * rb) / kFp8Block, wb - 1)) * nk);
#pragma unroll
    for (int j = 0; j < WB; ++j)
#pragma unroll
      for (int d = 0; d < kThinRun; ++d) s[j][d] = p[(int64_t)j * (wb / 2) * nk + min(kb0 + s0 + d, nk - 1)];
  };
  int i = t0 / tiles_per, n0 = (t0 % tiles_per) * width, have = -1, row0 = 0, rows = 0;
  int e_next = __builtin_amdgcn_readfirstlane((int)tab.thin[i]), e = e_next;
  scales(sw_next, e, n0, 0);
  for (int t = t0; t < t1; ++t) {
    if (i != have) {
      e = e_next;
      row0 = __builtin_amdgcn_readfirstlane(tab.rows[e]);
      rows = __builtin_amdgcn_readfirstlane(tab.rows[e + 1] - row0);
    }
#pragma unroll
    for (int j = 0; j < WB; ++j)
#pragma unroll
      for (int d = 0; d < kThinRun; ++d) sw[j][d] = sw_next[j][d];
    if (t + 1 < t1) {
      const bool on = n0 + width < cols;   // the next tile is of the same expert
      if (!on) e_next = __builtin_amdgcn_readfirstlane((int)tab.thin[i + 1]);
      scales(sw_next, e_next, on ? n0 + width : 0, 0);
    }
    v4f acc[MB][WB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int j = 0; j < WB; ++j) acc[m][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < per; s0 += kThinRun) {
      if (s0 != 0) scales(sw, e, n0, s0);
      if (i != have || per > kThinRun) {
        // the rows' k-blocks of this run, in the matrix instruction's layout
        const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(g.a + (int64_t)row0 * K), (short)0, rows * K, 0x00020000);
        const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<float*>(g.a_scale + (int64_t)row0 * nk), (short)0, rows * nk * 4, 0x00020000);
#pragma unroll
        for (int d = 0; d < kThinRun; ++d) {
          const int b = s0 + d < per ? kb0 + s0 + d : nk;
          const unsigned k0 = (unsigned)b * kFp8Block + 16u * quad, k1 = k0 + 64u;
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            const int row = 16 * m + r16;
            const unsigned at = (unsigned)(row * K);
            tok[d][m] = join(__builtin_amdgcn_raw_buffer_load_b128(ra, k0 < (unsigned)K ? at + k0 : kPastEnd, 0, 0),
                             __builtin_amdgcn_raw_buffer_load_b128(ra, k1 < (unsigned)K ? at + k1 : kPastEnd, 0, 0));
            sa[d][m] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                                     rq, b < nk ? (unsigned)(row * nk + b) * 4u : kPastEnd, 0, 0));
          }
        }
      }
#pragma unroll
      for (int d = 0; d < kThinRun; ++d) {
        if (s0 + d < per) {
          // vmcnt: at most the loads of the other slots are out
          __builtin_amdgcn_s_waitcnt(0x0F70 | ((kSlots - 1) * kLoads));
          v8i w[WB];
#pragma unroll
          for (int j = 0; j < WB; ++j) w[j] = lds_get2(f0 + read + j * 2048, f1 + read + j * 2048);
          read = read + kSlot == kSlots * kSlot ? 0 : read + kSlot;
          fetch();
#pragma unroll
          for (int j = 0; j < WB; ++j) {
            const float f = kb0 + s0 + d < nk ? sw[j][d] : 0.f;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
              const v4f p = mfma_block(w[j], tok[d][m]);
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[m][j][r] = __builtin_fmaf(p[r], sa[d][m] * f, acc[m][j][r]);
            }
          }
        }
      }
      have = i;
    }
    // join the runs of k-blocks: wavefront ob < rs sums those of block ob
#pragma unroll
    for (int m = 0; m < MB; ++m) {
#pragma unroll
      for (int j = 0; j < WB; ++j) lds_put(sm.red + ((wave * WB + j) * 64 + lane) * 16, acc[m][j]);
      lds_barrier();
      if (wave < rs) {
        v4f sum[WB];
#pragma unroll
        for (int j = 0; j < WB; ++j) sum[j] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < ks; ++k) {
          const unsigned at = sm.red + ((wave * ks + k) * WB * 64 + lane) * 16;
          const v8i p = lds_get2(at, at + (WB - 1) * 1024);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sum[0][r] += __int_as_float(p[r]);
            if (GLU) sum[WB - 1][r] += __int_as_float(p[4 + r]);
          }
        }
        const int row = 16 * m + r16, col = n0 + 16 * wave + 4 * quad;
        if (GLU) {
#pragma unroll
          for (int r = 0; r < 4; ++r) sum[0][r] = gmm_silu(sum[0][r]) * sum[WB - 1][r];
          if (blocks) lds_put(sm.g + (row * kLineG + col % kFp8Block) * 4, sum[0]);
          else if (row < rows) *reinterpret_cast<v4f*>(g.g + (int64_t)(row0 + row) * cols + col) = sum[0];
        } else if (row < rows && col < Nw) {
          *reinterpret_cast<v4b*>(g.y + (int64_t)(row0 + row) * Nw + col) = __builtin_convertvector(sum[0], v4b);
        }
      }
      lds_barrier();   // the sums have been read, SwiGLU's outputs are there
    }
    if (blocks && (n0 + width) % kFp8Block == 0) {
      static_assert(kThinRows * 16 == kGmmThreads, "a thread for 8 of the outputs");
      // row r = thread / 16, 8 columns per thread (overwritten only behind the next tile's first barrier)
      const int r = threadIdx.x >> 4, u = threadIdx.x & 15;
      const unsigned at = sm.g + (r * kLineG + 8 * u) * 4;
      const v8i v = lds_get2(at, at + 16);
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, (uint32_t)v[k] & 0x7FFFFFFFu);
      const Fp8Scaler f(row16_max(m));
      if (r < rows) {
        const int64_t q = (int64_t)(row0 + r) * (cols / kFp8Block) + n0 / kFp8Block;
        auto at8 = [&](int k) { return __int_as_float(v[k]); };
        reinterpret_cast<uint2*>(g.q)[q * 16 + u] =
            uint2{f.codes4(at8(0), at8(1), at8(2), at8(3)), f.codes4(at8(4), at8(5), at8(6), at8(7))};
        if (u == 0) g.q_scale[q] = f.scale;
      }
    }
    n0 += width;
    if (n0 >= cols) {
      n0 = 0;
      ++i;
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // no direct load into LDS is left in flight
}

// ks: at least 6 k-blocks per wavefront, and as many tiles as workgroups.
__device__ __forceinline__ int thin_split(const Gmm& g, int experts, int cols, bool blocks) {
  int ks = g.nk >= 48 ? 8 : g.nk >= 24 ? 4 : g.nk >= 12 ? 2 : 1;
  if (!blocks)
    while (ks < kGmmWaves && experts * ((cols + 128 / ks - 1) / (128 / ks)) < (int)gridDim.x) ks *= 2;
  return ks;
}

// ---------------------------------------------------------------------------
// Experts with more rows: tiles of BM = 32 to 256 rows x 256 weight rows (SwiGLU:
// 128 gate rows and the 128 up rows that go with them), one workgroup of eight
// wavefronts per CU walking tiles.  Each k-block of 128 is one stage, loaded
// global -> LDS directly into a ring of S stages while earlier ones are
// multiplied.  Wavefront (wt, wn) holds token blocks 2 i + wt (16 rows each, so
// that a short tile's blocks are shared) x 64 weight rows.
//
// LDS: chunk c (16 bytes) of row r sits at chunk c ^ ((r / 2) & 7) of the row's
// 128 bytes, so that 16 rows read at one chunk cover all banks.  A direct load
// writes lane l's 16 bytes at base + 16 l: eight rows per wavefront load, lane
// l taking row l / 8 and the chunk that belongs in slot l % 8.
//
// The scales sa[row][b] sw[.][b] of two periods of k-blocks lie behind the
// ring: thread (row, weight half, group) loads, multiplies and stores those of
// two k-blocks a period.  Tiles of 64 and 32 rows have threads for 8 and 16
// k-blocks (a load of 32 rows takes the address unit 27 ns; taken by every
// wavefront at every second k-block they cost a stage of 32 rows 0.1 of its 0.75
// us).
//
// The direct loads take their LDS addresses as numbers, and the waits for them
// are written out (a stage's before the barrier that opens it): told the array,
// the compiler would make every LDS read wait for every direct load.
// ---------------------------------------------------------------------------
constexpr int kWideW = 256;   // weight rows of a tile
constexpr int wide_stage(int BM) { return (BM + kWideW) * kFp8Block; }
constexpr int kWideScales = 8192;   // bytes of scales behind the ring
constexpr int wide_bytes(int BM, int S) { return S * wide_stage(BM) + kWideScales; }
// 128-row tiles take three stages where the experts' table leaves that much LDS.
constexpr int kLdsDeep = wide_bytes(128, 3), kLdsFlat = wide_bytes(256, 2);
static_assert(kLdsFlat >= wide_bytes(32, 3) && kLdsFlat >= wide_bytes(64, 3) && kLdsFlat >= wide_bytes(128, 2) &&
                  kLdsDeep >= wide_bytes(32, 4) && kLdsDeep >= kLdsFlat, "LDS of the tiles");

struct WideTile {
  int e, row0, rows, n0;   // n0: first weight row (SwiGLU: first output column)
};

// The k loop: acc[i][j] = token block 2 i + wt times weight block j of the
// wavefront.  NB: token blocks computed (the others hold no rows).
template <bool GLU, int BM, int S, int NB>
__device__ __forceinline__ void wide_kloop(const Gmm& g, const WideTile& t, uint8_t* smem, v4f (&acc)[BM / 32][4]) {
  constexpr int kStage = wide_stage(BM), kRing = S * kStage;
  constexpr int kTokenBytes = BM * kFp8Block;
  constexpr int kTokenLoads = (BM + 63) / 64;   // direct loads of token rows per wavefront and stage (8 rows each)
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave >> 2, wn = wave & 3;
  const int K = g.K, nk = g.nk, Nw = g.Nw;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.a + (int64_t)t.row0 * K), (short)0, t.rows * K, 0x00020000);
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(g.a_scale + (int64_t)t.row0 * nk), (short)0, t.rows * nk * 4, 0x00020000);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.w + ((int64_t)t.e * Nw + t.n0) * K), (short)0, (Nw - t.n0) * K, 0x00020000);

  // ---- loads ----
  unsigned vo[2], chunk[2];   // lane part of a load of eight rows, by the parity of its place
#pragma unroll
  for (int par = 0; par < 2; ++par) {
    chunk[par] = (unsigned)(((lane & 7) ^ ((4 * par + (lane >> 4)) & 7)) << 4);
    vo[par] = (unsigned)((lane >> 3) * K) + chunk[par];
  }
  const unsigned up = GLU && wave >= 4 ? (unsigned)((Nw / 2 - kWideW / 2) * K) : 0u;   // weight rows 128 .. 255
  // Direct loads of k-block b, of kLoads in kParts parts.  (No branches here
  // and below: they would split the schedule.)
  constexpr int kLoads = kTokenLoads + 4;
  constexpr bool kFine = NB <= 2;   // a part behind each matrix instruction
  constexpr int kParts = kFine ? 4 * NB : NB / 2 + 1, kPart = (kLoads + kParts - 1) / kParts;
  const unsigned lds = lds_at(smem);
  auto dma = [&](int at, int b, int part) {   // at: the stage's place in the ring
    unsigned v[2];
    const unsigned k0 = (unsigned)b * kFp8Block;
#pragma unroll
    for (int par = 0; par < 2; ++par) v[par] = k0 + chunk[par] < (unsigned)K ? vo[par] : kPastEnd;   // zeros past K
#pragma unroll
    for (int q = part * kPart; q < min(kLoads, (part + 1) * kPart); ++q) {
      if (q < 4) {
        const int blk = 4 * wave + q;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(size_t)(lds + at + kTokenBytes + blk * 1024), 16, v[q & 1],
                                                 k0 + (unsigned)(8 * blk * K) + up, 0, 0);
      } else {
        const int blk = (kTokenLoads * wave + q - 4) & (BM / 8 - 1);   // (BM = 32: two wavefronts load the same)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(size_t)(lds + at + blk * 1024), 16, v[blk & 1],
                                                 k0 + (unsigned)(8 * blk * K), 0, 0);
      }
    }
  };
  // ---- scales of the kPeriod k-blocks from b, a multiple of kPeriod: two of
  // them for thread (row, weight half, group) ----
  // (The larger tiles take the two next k-blocks every second stage, 128 rows
  // twice: a condition in their loop makes the compiler spill.)
  constexpr int kGroups = BM < 128 ? kGmmThreads / (2 * BM) : 1, kPeriod = 2 * kGroups;
  static_assert(2 * kPeriod * 2 * BM * (int)sizeof(float) <= kWideScales, "two periods of scales");
  const int wb = (Nw + kFp8Block - 1) / kFp8Block;
  const int sgroup = tid % kGroups, half = tid / kGroups & 1, srow = tid / (2 * kGroups) & (BM - 1);
  const int wblock = t.n0 / kFp8Block;
  const unsigned wnext = (unsigned)((GLU ? wb / 2 : min(1, wb - 1 - wblock)) * nk) * 4u;   // from the first half's scales
  const __amdgpu_buffer_rsrc_t rv = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(g.w_scale + ((int64_t)t.e * wb + wblock) * nk), (short)0, (int)wnext + nk * 4, 0x00020000);
  v2f sa, sw;
  auto scale_load = [&](int b) {
    sa = __builtin_bit_cast(v2f, __builtin_amdgcn_raw_buffer_load_b64(rs, (unsigned)(srow * nk + 2 * sgroup) * 4u, (unsigned)b * 4u, 0));
    sw = __builtin_bit_cast(v2f, __builtin_amdgcn_raw_buffer_load_b64(rv, (half ? wnext : 0u) + 8u * (unsigned)sgroup, (unsigned)b * 4u, 0));
  };
  float* const sc = reinterpret_cast<float*>(smem + kRing);   // [2 kPeriod][2 weight halves][BM], k-block b at b % (2 kPeriod)
  auto scale_store = [&](int b) {
    const int mine = b + 2 * sgroup;
    float* p = sc + (mine & (2 * kPeriod - 1)) * 2 * BM + half * BM + srow;
    p[0] = mine < nk ? sa[0] * sw[0] : 0.f;
    p[2 * BM] = mine + 1 < nk ? sa[1] * sw[1] : 0.f;
  };

  // ---- fragments ----
  const int r16 = lane & 15, quad = lane >> 4;
  const int key = (lane >> 1) & 7;
  const int f0 = r16 * kFp8Block + ((quad ^ key) << 4), f1 = r16 * kFp8Block + (((4 + quad) ^ key) << 4);
  auto wrow = [&](int j) {   // first LDS weight row of the wavefront's block j
    if (GLU) return (j < 2 ? 0 : kWideW / 2 - 32) + 32 * wn + 16 * j;
    return 64 * wn + 16 * j;
  };
  auto wfrag = [&](int at, int j) {
    const uint8_t* p = smem + at + kTokenBytes + wrow(j) * kFp8Block;
    return join(*reinterpret_cast<const v4i*>(p + f0), *reinterpret_cast<const v4i*>(p + f1));
  };
  auto tfrag = [&](int at, int i) {
    const uint8_t* p = smem + at + (32 * i + 16 * wt) * kFp8Block;
    return join(*reinterpret_cast<const v4i*>(p + f0), *reinterpret_cast<const v4i*>(p + f1));
  };
  const float* const my_sc = sc + (GLU ? 0 : (wn >> 1) * BM) + 16 * wt + r16;
  struct Sc {
    float s[GLU ? 2 : 1];
  };
  auto scale = [&](int b, int i) {
    const float* p = my_sc + (b & (2 * kPeriod - 1)) * 2 * BM + 32 * i;
    Sc s;
#pragma unroll
    for (int h = 0; h < (GLU ? 2 : 1); ++h) s.s[h] = p[h * BM];
    return s;
  };
  auto add = [&](v4f& c, const v4f& p, float f) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c[r] = __builtin_fmaf(p[r], f, c[r]);
  };

  // Stages 0 .. S - 2 are loaded ahead, and the first part of stage S - 1.
  constexpr int kAhead = 0x0F70 | (((S - 2) * kLoads) & 15) | ((((S - 2) * kLoads) >> 4) << 14);   // vmcnt of S - 2 stages
  scale_load(0);
#pragma unroll
  for (int d = 0; d < S - 1; ++d)
#pragma unroll
    for (int part = 0; part < kParts; ++part) dma(d * kStage, d, part);
  scale_store(0);
  __builtin_amdgcn_s_waitcnt(kAhead);   // this wavefront's loads of stage 0 have landed
  lds_barrier();
#pragma unroll
  for (int part = 0; part < (kFine ? 4 : 1); ++part) dma((S - 1) * kStage, S - 1, part);
  scale_load(kPeriod);
  v8i w[4], tok = tfrag(0, 0), tok_next;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = wfrag(0, j);
  Sc s_prev{}, s_cur = scale(0, 0), s_next;
  v4f p[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = v4f{0.f, 0.f, 0.f, 0.f};
  // Each step issues one matrix instruction and adds the result of the one
  // three steps before, across token blocks and stages.
  int cur = 0, nxt = kStage, last = (S - 1) * kStage;   // places of k-blocks b, b + 1, b + S - 1
  auto stage = [&](int b, bool odd) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (!kFine && i + 1 < kParts) dma(last, b + S - 1, i + 1);   // (all at once they would hold up the products)
      if (i + 1 < NB) {
        tok_next = tfrag(cur, i + 1);
        s_next = scale(b, i + 1);
      } else {
        __builtin_amdgcn_s_waitcnt(kAhead);   // this wavefront's loads of k-block b + 1 have landed
        if (odd && (b + 1) % kPeriod == 0) scale_store(b + 1);   // (loaded a period before)
        lds_barrier();
        if (!kFine) dma(cur, b + S, 0);
        if (odd && (b + 1) % kPeriod == 0) scale_load(b + 1 + kPeriod);
        tok_next = tfrag(nxt, 0);   // (after the last stage: read, never used)
        s_next = scale(b + 1, 0);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = mfma_block(w[j], tok);
        if (kFine) {
          if (i + 1 == NB) dma(cur, b + S, j);
          else dma(last, b + S - 1, 4 * (i + 1) + j);
        }
        if (i + 1 == NB) w[j] = wfrag(nxt, j);
        if (j < 3) add(acc[(i + NB - 1) % NB][j + 1], p[j + 1], s_prev.s[GLU ? (j + 1) >> 1 : 0]);
        else add(acc[i][0], p[0], s_cur.s[0]);
        __builtin_amdgcn_sched_barrier(0);
      }
      tok = tok_next;
      s_prev = s_cur;
      s_cur = s_next;
    }
    last = cur;
    cur = nxt;
    nxt = nxt + kStage == kRing ? 0 : nxt + kStage;
  };
  for (int b = 0; b < nk; b += 2) {   // (past an odd last k-block comes one of zeros)
    stage(b, false);
    stage(b + 1, true);
  }
#pragma unroll
  for (int j = 1; j < 4; ++j) add(acc[NB - 1][j], p[j], s_prev.s[GLU ? j >> 1 : 0]);
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): the loads past the last stage (of zeros) have landed too
}

// One tile: the k loop, then the outputs through LDS as whole rows.
template <bool GLU, int BM, int S>
__device__ __forceinline__ void wide_tile(const Gmm& g, const WideTile& t, uint8_t* smem) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave >> 2, wn = wave & 3;
  const int r16 = lane & 15, quad = lane >> 4;
  v4f acc[BM / 32][4];
#pragma unroll
  for (int i = 0; i < BM / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  if constexpr (BM <= 64) wide_kloop<GLU, BM, S, BM / 32>(g, t, smem, acc);
  else if (t.rows > BM * 3 / 4) wide_kloop<GLU, BM, S, BM / 32>(g, t, smem, acc);
  else if (t.rows > BM / 2) wide_kloop<GLU, BM, S, (BM * 3 / 4 + 31) / 32>(g, t, smem, acc);
  else if (t.rows > BM / 4) wide_kloop<GLU, BM, S, BM / 64>(g, t, smem, acc);
  else wide_kloop<GLU, BM, S, (BM + 127) / 128>(g, t, smem, acc);
  __syncthreads();   // every wavefront has left the ring
  if (GLU) {
    // g = silu(gate) * up (columns 32 wn + 16 j + 4 quad + r), its row maxima
    // over the 128 columns, and the codes
    uint32_t* top = reinterpret_cast<uint32_t*>(smem + BM * kFp8Block);   // [4][BM]
#pragma unroll
    for (int i = 0; i < BM / 32; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[i][j][r] = gmm_silu(acc[i][j][r]) * acc[i][j + 2][r];
          m = max(m, abs_bits(acc[i][j][r]));
        }
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      if (quad == 0) top[wn * BM + 32 * i + 16 * wt + r16] = m;
    }
    __syncthreads();
    const int nb2 = g.Nw / 2 / kFp8Block;
#pragma unroll
    for (int i = 0; i < BM / 32; ++i) {
      const int row = 32 * i + 16 * wt + r16;
      uint32_t m = top[row];
#pragma unroll
      for (int w = 1; w < 4; ++w) m = max(m, top[w * BM + row]);
      const Fp8Scaler f(m);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int unit = 2 * wn + j;   // 16 columns
        *reinterpret_cast<uint32_t*>(smem + row * kFp8Block + ((unit ^ (row & 7)) << 4) + 4 * quad) =
            f.codes4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
      }
      if (wn == 0 && quad == 0 && row < t.rows) g.q_scale[(int64_t)(t.row0 + row) * nb2 + t.n0 / kFp8Block] = f.scale;
    }
    __syncthreads();
    for (int r = tid >> 3; r < t.rows; r += kGmmThreads / 8) {
      const int unit = tid & 7;
      *reinterpret_cast<v4u*>(g.q + (int64_t)(t.row0 + r) * (g.Nw / 2) + t.n0 + 16 * unit) =
          *reinterpret_cast<const v4u*>(smem + r * kFp8Block + ((unit ^ (r & 7)) << 4));
    }
  } else {
#pragma unroll
    for (int i = 0; i < BM / 32; ++i) {
      const int row = 32 * i + 16 * wt + r16;
      uint8_t* line = smem + row * 512;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int unit = 8 * wn + 2 * j + (quad >> 1);   // 8 columns
        *reinterpret_cast<v4b*>(line + ((unit ^ (row & 31)) << 4) + 8 * (quad & 1)) =
            __builtin_convertvector(acc[i][j], v4b);
      }
    }
    __syncthreads();
    const int unit = tid & 31, col = t.n0 + 8 * unit;
    if (col < g.Nw)
      for (int r = tid >> 5; r < t.rows; r += kGmmThreads / 32)
        *reinterpret_cast<v4u*>(g.y + (int64_t)(t.row0 + r) * g.Nw + col) =
            *reinterpret_cast<const v4u*>(smem + r * 512 + ((unit ^ (r & 31)) << 4));
  }
  __syncthreads();   // the ring is free
}

// Tile number -> place.  The m-tiles of an expert run in chunks of up to 8,
// and a chunk's tiles in groups of h m-tiles x 32 / h n-tiles, m fastest, so
// that the about 32 tiles an XCD runs at a time share rows and weights in its
// L2.
__device__ __forceinline__ WideTile wide_place(const Gmm& g, const GmmTable& tab, int t, int nn, int BM, int cols) {
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

template <bool GLU, int BM, int S>
__device__ __forceinline__ void wide_walk(const Gmm& g, const GmmTable& tab, uint8_t* smem) {
  constexpr int kCols = GLU ? kWideW / 2 : kWideW;
  const int nn = ((GLU ? g.Nw / 2 : g.Nw) + kCols - 1) / kCols;
  const int T = tab.tiles[g.L] * nn;
  for (int t = wide_line(); t < T; t += gridDim.x)
    wide_tile<GLU, BM, S>(g, wide_place(g, tab, t, nn, BM, kCols), smem);
}

// What a k-block of a tile of 256, 128, 64 and 32 rows takes, in tenths of a
// microsecond (4096, 2048, 1024 and 512 rows x 4096 x 7168, so that 256
// workgroups have one tile each: 118, 73, 48 and 39 us, the plan of the tiles 4
// of them slower than now).  Both sides of the choice, likewise: those 512 rows take 45 us in tiles of 64 rows and 65 us in tiles of
// 128; 512 x 7168 x 2048 takes 21 us in 224 tiles of 64 rows and 27 us in two
// rounds of 32-row tiles; 2048 x 7168 x 2048 41 us in tiles of 256 rows, 47 us
// in two rounds of 128 and 56 us in four of 64.
constexpr int kCost256 = 20, kCost128 = 12, kCost64 = 8, kCost32 = 6;

// One workgroup per CU: the wide experts' tiles, then the thin experts'.
// DEEP: the LDS holds three stages of 128-row tiles.
template <bool GLU, bool DEEP>
__global__ __launch_bounds__(kGmmThreads) void k_gmm(Gmm g) {
  extern __shared__ int gmm_table[];
  __shared__ __attribute__((aligned(16))) uint8_t smem[DEEP ? kLdsDeep : kLdsFlat];
  __shared__ int64_t wave_total[kGmmWaves];
  GmmTable tab{gmm_table, gmm_table + g.L + 1, reinterpret_cast<uint16_t*>(gmm_table + 2 * (g.L + 1)), 0};
  if (g.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *g.status = mdc_device_status{0, 0, 0, 0};
  gmm_rows<kGmmThreads>(g, tab.rows, wave_total);
  constexpr int kCols = GLU ? kWideW / 2 : kWideW;
  const int nn = ((GLU ? g.Nw / 2 : g.Nw) + kCols - 1) / kCols;
  const int G = gridDim.x;
  int wide = gmm_tiles(g, tab, 256, wave_total) * nn;
  if (wide != 0) {
    // Tiles of 256, 128 or 64 rows, whichever rounds of tiles take less time:
    // large ones do more products per byte and stage, small ones fill the CUs.
    int best = 256, cost = kCost256 * ((wide + G - 1) / G), count[3];
    gmm_tile_counts(g, tab, count);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = (i == 0 ? kCost128 : i == 1 ? kCost64 : kCost32) * ((count[i] * nn + G - 1) / G);
      if (c < cost) {
        best = 128 >> i;
        cost = c;
      }
    }
    if (best != 256) wide = gmm_tiles(g, tab, best, wave_total) * nn;
    if (best == 32) wide_walk<GLU, 32, DEEP ? 4 : 3>(g, tab, smem);
    else if (best == 64) wide_walk<GLU, 64, 3>(g, tab, smem);
    else if (best == 128) wide_walk<GLU, 128, DEEP ? 3 : 2>(g, tab, smem);
    else wide_walk<GLU, 256, 2>(g, tab, smem);
  }
  if (tab.n_thin != 0) {
    __syncthreads();   // smem is free
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kRings = kGmmWaves * kThinRing;
    static_assert(kRings + kGmmWaves * 2 * 1024 + kThinRows * kLineG * 4 <= kLdsFlat, "LDS of the thin tiles");
    const ThinSmem sm{lds_at(smem) + wave * kThinRing, lds_at(smem) + kRings,
                      lds_at(smem) + kRings + kGmmWaves * 2 * 1024};
    thin_walk<GLU>(g, tab, wide, thin_split(g, tab.n_thin, GLU ? g.Nw / 2 : g.Nw, GLU && !g.split), sm);
  }
}

// ---------------------------------------------------------------------------
// Rows to fp8: one scale per 128 columns, 16 lanes x 8 values per block.  Bound:
// memory (16384 x 7168 bf16 62 to 65 us, 5.5 to 5.7 TB/s; in a decode step, 256
// rows, 5 us, of which an empty launch is 1.8).
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;

// rows in use: min(sum of the counts, A)
__device__ __forceinline__ int64_t rows_in_use(const int64_t* nums, int L, int64_t A) {
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  for (int e = lane; e < L; e += 64) total += min(max(nums[e], (int64_t)0), A);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o, 64);
  return min(total, A);
}

// x [rows][128 nb] bf16 -> q, s.
__global__ __launch_bounds__(kQuantThreads) void k_quant_fp8_rows(const v4u* __restrict__ x, uint2* __restrict__ q,
                                                                  float* __restrict__ s,
                                                                  const int64_t* __restrict__ nums, int L, int64_t A,
                                                                  int nb) {
  const int64_t n = rows_in_use(nums, L, A) * nb * 16;   // vectors of 8
  for (int64_t i = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x; i < (n + 63) / 64 * 64;
       i += (int64_t)gridDim.x * kQuantThreads) {
    const v4u v = i < n ? x[i] : v4u{0u, 0u, 0u, 0u};
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = max(m, max(abs_bits(bf16_lo(v[w])), abs_bits(bf16_hi(v[w]))));
    const Fp8Scaler f(row16_max(m));
    if (i < n) {
      q[i] = uint2{f.codes4(bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])),
                   f.codes4(bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3]))};
      if ((i & 15) == 0) s[i >> 4] = f.scale;
    }
  }
}

// g (fp32) -> q, s of the thin experts' rows.  One workgroup per (expert, row),
// strided.
__global__ __launch_bounds__(kQuantThreads) void k_quant_fp8_thin(Gmm g) {
  extern __shared__ int gmm_table[];
  __shared__ int64_t wave_total[kQuantThreads / 64];
  int* rows = gmm_table;
  gmm_rows<kQuantThreads>(g, rows, wave_total);
  const int nvec = g.Nw / 2 / 8;   // a multiple of 16
  for (int m = blockIdx.x; m < g.L * kThinRows; m += gridDim.x) {
    const int e = m / kThinRows, in = m - e * kThinRows;
    const int count = rows[e + 1] - rows[e], row = rows[e] + in;
    if (count > kThinRows || in >= count) continue;
    const v4f* src = reinterpret_cast<const v4f*>(g.g + (int64_t)row * (g.Nw / 2));
    for (int i = threadIdx.x; i < (nvec + 63) / 64 * 64; i += kQuantThreads) {
      const v4f z = {0.f, 0.f, 0.f, 0.f};
      const v4f a = i < nvec ? src[2 * i] : z, b = i < nvec ? src[2 * i + 1] : z;
      uint32_t mx = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) mx = max(mx, max(abs_bits(a[r]), abs_bits(b[r])));
      const Fp8Scaler f(row16_max(mx));
      if (i < nvec) {
        reinterpret_cast<uint2*>(g.q)[(int64_t)row * nvec + i] =
            uint2{f.codes4(a[0], a[1], a[2], a[3]), f.codes4(b[0], b[1], b[2], b[3])};
        if ((i & 15) == 0) g.q_scale[(int64_t)row * (nvec >> 4) + (i >> 4)] = f.scale;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
unsigned device_cus() {
  int dev = 0, cus = 256;
  if (hipGetDevice(&dev) == hipSuccess) (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  return (unsigned)cus;
}

// Whether thin experts' SwiGLU outputs go through memory in fp32 and a launch
// that quantises them: where the 128-column blocks are too few for the CUs, and
// the capacity says that thin experts are what there is (which experts are thin
// is known on the device only, and g has a row for each of the capacity's).  FFN
// of 7168 and 4096 with 8 rows an expert, whole blocks : split, in us: 16 blocks 74
// : 33, 64 blocks 82 : 52, 128 blocks 98 : 83, 192 blocks 119 : 118, 256 blocks 138
// : 142, 384 blocks 221 : 208 (one and a half rounds of 256 workgroups; a larger
// bound would split the 256 blocks too).  A capacity above kSplitRows rows an expert
// takes whole blocks at any number of them.
constexpr int kSplitBlocks = 192, kSplitRows = 128;
bool gmm_split(int64_t A, int64_t L, int64_t cols) {
  return L * (cols / kFp8Block) < kSplitBlocks && A <= L * kSplitRows;
}

constexpr size_t kLdsSize = 160 << 10;   // of a CU

template <bool GLU>
void launch_gmm(const Gmm& g, hipStream_t s) {
  const dim3 grid((device_cus() + 7) / 8 * 8), block(kGmmThreads);
  const size_t table = gmm_table_bytes(g.L);
  if (table + kLdsDeep + 256 <= kLdsSize)   // (256: the plan's few words)
    hipLaunchKernelGGL((k_gmm<GLU, true>), grid, block, table, s, g);
  else hipLaunchKernelGGL((k_gmm<GLU, false>), grid, block, table, s, g);
}

constexpr int kMaxK = 1 << 22;   // the rows of a tile are addressed with 32-bit offsets

mdc_status check_gmm(int64_t A, int32_t L, int32_t n, int32_t k) {
  if (A < 0 || L < 1 || n < 1 || k < 1 || n % 8 != 0 || k % 16 != 0) return MDC_ERR_INVALID;
  if (L > MDC_MAX_LOCAL_EXPERTS || A > INT32_MAX || (int64_t)n * k > INT32_MAX || k > kMaxK) return MDC_ERR_UNSUPPORTED;
  if ((A / kThinRows + L + 1) * ((n + 15) / 16) > INT32_MAX - 65536) return MDC_ERR_UNSUPPORTED;
  return MDC_OK;
}

// Workspace: [status block][q1][s1][q2][s2][g, where thin experts split k].
struct Ffn8Plan {
  int64_t A;
  int H, N, L;
  size_t off_q1, off_s1, off_q2, off_s2, off_g, bytes;
};

Ffn8Plan make_ffn8_plan(const mdc_shape* sh, int inter_n) {
  Ffn8Plan f;
  f.A = sh->capacity;
  f.H = sh->hidden;
  f.N = inter_n;
  f.L = sh->num_experts / sh->world;
  const size_t A = (size_t)f.A, H = (size_t)f.H, I = (size_t)f.N / 2;
  f.off_q1 = MDC_STATUS_BYTES;
  f.off_s1 = f.off_q1 + round_up(A * H, 256);
  f.off_q2 = f.off_s1 + round_up(A * (H / kFp8Block) * 4, 256);
  f.off_s2 = f.off_q2 + round_up(A * I, 256);
  f.off_g = f.off_s2 + round_up(A * (I / kFp8Block) * 4, 256);
  f.bytes = f.off_g + (gmm_split(f.A, f.L, I) ? round_up(A * I * 4, 256) : 0);
  return f;
}

mdc_status check_ffn8(const mdc_shape* sh, int inter_n) {
  mdc_status st = check_shape(sh);
  if (st != MDC_OK) return st;
  if (inter_n <= 0) return MDC_ERR_INVALID;
  if (inter_n % 256 != 0 || sh->hidden % kFp8Block != 0) return MDC_ERR_UNSUPPORTED;
  const int32_t L = sh->num_experts / sh->world;
  st = check_gmm(sh->capacity, L, inter_n, sh->hidden);
  return st != MDC_OK ? st : check_gmm(sh->capacity, L, sh->hidden, inter_n / 2);
}

mdc_status ffn8_impl(const mdc_shape* shape, int32_t inter_n, const void* expand_x, const void* expand_q,
                     const float* scales, const int64_t* nums, const void* w1, const float* w1_scale, const void* w2,
                     const float* w2_scale, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  const mdc_status st = check_ffn8(shape, inter_n);
  if (st != MDC_OK) return st;
  const Ffn8Plan f = make_ffn8_plan(shape, inter_n);
  if (f.A == 0) return MDC_OK;
  if ((expand_x == nullptr && (expand_q == nullptr || scales == nullptr)) || nums == nullptr || w1 == nullptr ||
      w1_scale == nullptr || w2 == nullptr || w2_scale == nullptr || y == nullptr || workspace == nullptr)
    return MDC_ERR_NULLPTR;
  if (!aligned16(expand_x) || !aligned16(expand_q) || !aligned4(scales) || !aligned8(nums) || !aligned16(w1) ||
      !aligned4(w1_scale) || !aligned16(w2) || !aligned4(w2_scale) || !aligned16(y) || !aligned16(workspace))
    return MDC_ERR_INVALID;
  if (workspace_bytes < f.bytes) return MDC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  mdc_device_status* status = reinterpret_cast<mdc_device_status*>(ws);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned cus = device_cus();
  (void)hipGetLastError();
  const uint8_t* q1 = static_cast<const uint8_t*>(expand_q);
  if (expand_x != nullptr) {
    uint2* q = reinterpret_cast<uint2*>(ws + f.off_q1);
    float* s1 = reinterpret_cast<float*>(ws + f.off_s1);
    hipLaunchKernelGGL(k_quant_fp8_rows, dim3(cus * 8), dim3(kQuantThreads), 0, s, static_cast<const v4u*>(expand_x),
                       q, s1, nums, f.L, f.A, f.H / kFp8Block);
    q1 = reinterpret_cast<const uint8_t*>(q);
    scales = s1;
  }
  uint8_t* q2 = reinterpret_cast<uint8_t*>(ws + f.off_q2);
  float* s2 = reinterpret_cast<float*>(ws + f.off_s2);
  const Gmm g1{q1, scales, nums, static_cast<const uint8_t*>(w1), w1_scale, nullptr,
               reinterpret_cast<float*>(ws + f.off_g), q2, s2, status, (int)f.A, f.L, f.N, f.H, f.H / kFp8Block,
               gmm_split(f.A, f.L, f.N / 2)};
  launch_gmm<true>(g1, s);
  if (g1.split)
    hipLaunchKernelGGL(k_quant_fp8_thin, dim3((unsigned)min((int64_t)f.L * kThinRows, (int64_t)cus * 8)),
                       dim3(kQuantThreads), ((size_t)f.L + 1) * sizeof(int), s, g1);
  const Gmm g2{q2, s2, nums, static_cast<const uint8_t*>(w2), w2_scale, static_cast<uint16_t*>(y), nullptr, nullptr, nullptr,
               nullptr, (int)f.A, f.L, f.H, f.N / 2, f.N / 2 / kFp8Block, 0};
  launch_gmm<false>(g2, s);
  return launched();
}

}  // namespace

extern "C" {

mdc_status mdc_gmm_fp8(int64_t capacity, int32_t experts, int32_t n, int32_t k, const void* a, const float* a_scale,
                       const int64_t* expert_token_nums, const void* w, const float* w_scale, void* y, void* stream) {
  const mdc_status st = check_gmm(capacity, experts, n, k);
  if (st != MDC_OK) return st;
  if (capacity == 0) return MDC_OK;
  if (a == nullptr || a_scale == nullptr || w == nullptr || w_scale == nullptr || y == nullptr ||
      (expert_token_nums == nullptr && experts != 1))
    return MDC_ERR_NULLPTR;
  if (!aligned16(a) || !aligned4(a_scale) || !aligned8(expert_token_nums) || !aligned16(w) || !aligned4(w_scale) ||
      !aligned16(y))
    return MDC_ERR_INVALID;
  (void)hipGetLastError();
  const Gmm g{static_cast<const uint8_t*>(a), a_scale, expert_token_nums, static_cast<const uint8_t*>(w), w_scale,
              static_cast<uint16_t*>(y), nullptr, nullptr, nullptr, nullptr, (int)capacity, experts, n, k,
              (k + kFp8Block - 1) / kFp8Block, 0};
  launch_gmm<false>(g, static_cast<hipStream_t>(stream));
  return launched();
}

mdc_status mdc_ffn_fp8_workspace(const mdc_shape* shape, int32_t inter_n, size_t* bytes) {
  if (bytes == nullptr) return MDC_ERR_NULLPTR;
  const mdc_status st = check_ffn8(shape, inter_n);
  if (st != MDC_OK) return st;
  *bytes = make_ffn8_plan(shape, inter_n).bytes;
  return MDC_OK;
}

mdc_status mdc_ffn_fp8(const mdc_shape* shape, int32_t inter_n, const void* expand_x, const int64_t* expert_token_nums,
                       const void* w1, const float* w1_scale, const void* w2, const float* w2_scale, void* y,
                       void* workspace, size_t workspace_bytes, void* stream) {
  return ffn8_impl(shape, inter_n, expand_x, nullptr, nullptr, expert_token_nums, w1, w1_scale, w2, w2_scale, y,
                   workspace, workspace_bytes, stream);
}

mdc_status mdc_ffn_fp8_quant_input(const mdc_shape* shape, int32_t inter_n, const void* expand_q,
                                   const float* dynamic_scales, const int64_t* expert_token_nums, const void* w1,
                                   const float* w1_scale, const void* w2, const float* w2_scale, void* y,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  return ffn8_impl(shape, inter_n, nullptr, expand_q, dynamic_scales, expert_token_nums, w1, w1_scale, w2, w2_scale, y,
                   workspace, workspace_bytes, stream);
}

}  // extern "C"
