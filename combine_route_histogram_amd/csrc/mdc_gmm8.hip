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
//
// Three ways in one launch, by an expert's rows and the call's tiles.  What bounds
// them: few rows, the weights' way from memory (256 rows of 30 experts x 4096 x 7168:
// 135 us, 6.5 TB/s); many, the matrix units at the clock that they leave (4096 x 4096
// x 7168: 100 us, 2.4 POP/s; 89 us without the stages' direct loads, 84 without LDS
// reads too; the library's product without scales 102); those between, the time from
// one k-block to the next; small calls, the launch and the plan (one row x 7168 x
// 2048: 9.4 us, 2.2 of them the weights at that rate).
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
// Thin experts.  A tile is one expert's rows times 16 rs output columns: wavefront
// (rb, kh) takes 16 weight rows of it over the kh-th of ks runs of k-blocks,
// rs ks = 8, and the runs' sums are joined through LDS.  A workgroup takes a run of
// consecutive tiles.
//
// The weights, which are all that memory has to bring, go global -> LDS directly,
// eight rows x 128 bytes per instruction, into a ring of each wavefront's own,
// kThin8Ring bytes ahead and on into the next tile.  They are read once: with the
// non-temporal policy such loads reach 6.8 TB/s, without it 6.0 (940 MB, tiles of
// 16 rows; the same for runs of 128 to 512 bytes and rings of 8 to 18 KB).  The
// expert's rows stay in registers from tile to tile, kThin8Run k-blocks of them.
//
// The border of 32 rows is that of two blocks of the instruction, for any number of
// experts; 32 : 33 rows each, in us: one expert x 4096 x 7168 12.7 : 20.4, four 24.1 :
// 25.5, 16 x 4096 x 2048 28.3 : 24.3, 8 x 2048 x 1024 11.2 : 8.8.
//
// LDS accesses are written out with their waits: the compiler would make each wait
// for every direct load in flight.
// ---------------------------------------------------------------------------
constexpr int kThin8Ring = 12288;   // bytes of a wavefront's ring
constexpr int kThin8Run = 8;        // k-blocks of rows in registers
constexpr int kThin8Direct = 16;    // most rows that are always loaded in the instruction's layout
constexpr int kThin8Nt = 2;         // cache policy: non-temporal

struct Thin8Smem {
  unsigned ring;   // this wavefront's, kThin8Ring bytes
  unsigned red;    // [2][8 wavefronts][2 row blocks][64] v4i
};

__device__ __forceinline__ void thin8_walk(const Gmm8& g, const GmmTable& tab, int wide, int cost16, int ks, const Thin8Smem& sm) {
  constexpr int MB = kThinBlocks, kSlot = 2048, kSlots = kThin8Ring / kSlot;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const int K = g.K, nk = g.nk, Nw = g.Nw;
  const int rs = kGmmWaves / ks, rb = wave / ks, kh = wave - rb * ks;
  const int per = (nk + ks - 1) / ks, kb0 = kh * per;
  const int width = 16 * rs, tiles_per = (Nw + width - 1) / width;
  // this workgroup's tiles: [t0, t1) of n_thin * tiles_per
  const int64_t T = (int64_t)tab.n_thin * tiles_per;
  const int cost = max(1, cost16 / rs);
  const int t0 = (int)thin_share(T, wide, cost, wide_line()), t1 = (int)thin_share(T, wide, cost, wide_line() + 1);
  if (t0 == t1) return;

  // ---- weights: tile by tile, step by step ----
  auto weights = [&](int i) {
    const int e = __builtin_amdgcn_readfirstlane((int)tab.thin[i]);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(g.w + (int64_t)e * Nw * K), (short)0, Nw * K, 0x00020000);
  };
  struct {
    int i, n, step, left;   // place of the expert in the list, first column, step, tiles to come
  } c = {t0 / tiles_per, (t0 % tiles_per) * width, 0, t1 - t0};
  __amdgpu_buffer_rsrc_t rw = weights(c.i);
  unsigned slot = 0;   // of the next load
  const int lrow = lane >> 3, key = (r16 >> 1) & 7;
  auto fetch = [&]() {
    const bool in = c.left > 0;
    const unsigned k0 = in ? (unsigned)min(kb0 + c.step, nk) * kGmm8Block : (unsigned)nk * kGmm8Block;
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // rows 8 h + lane / 8; the chunk whose place lane % 8 is
      const unsigned chunk = (unsigned)((lane & 7) ^ ((4 * h + (lrow >> 1)) & 7)) << 4;
      const int row = c.n + 16 * rb + 8 * h + lrow;
      const unsigned at = k0 + chunk < (unsigned)K && row < Nw ? (unsigned)row * (unsigned)K + k0 + chunk : kPastEnd;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(size_t)(sm.ring + slot + h * 1024), 16, at, 0, 0, kThin8Nt);
    }
    slot = slot + kSlot == kSlots * kSlot ? 0 : slot + kSlot;
    if (++c.step == per) {
      c.step = 0;
      --c.left;
      c.n += width;
      if (c.n >= Nw) {
        c.n = 0;
        if (c.left > 0) rw = weights(++c.i);
      }
    }
  };

  // ---- the expert's rows, which are on their way before the weights ----
  v8i tok[kThin8Run][MB];
  float sa[MB];
  int i = c.i, n0 = c.n, have = i, held = 0, e = 0, row0 = 0, rows = 0;
  auto expert = [&]() {
    e = __builtin_amdgcn_readfirstlane((int)tab.thin[i]);
    row0 = __builtin_amdgcn_readfirstlane(tab.rows[e]);
    rows = __builtin_amdgcn_readfirstlane(tab.rows[e + 1] - row0);
#pragma unroll
    for (int m = 0; m < MB; ++m) sa[m] = g.a_scale[row0 + min(16 * m + r16, rows - 1)];
  };
  // Their k-blocks s0 ... of the run, in the matrix instruction's layout.  Loaded in it,
  // lanes side by side take 16 bytes of different rows, and a load costs by its rows; of
  // many rows and k-blocks a row's 128 bytes are loaded by eight lanes, and place() turns
  // them.  Loaded so : turned, in us, 32 rows each: 16 experts x 4096 x 2048 31.3 : 28.3,
  // one x 4096 x 7168 14.0 : 12.7; 16 rows of it 11.7 : 12.3; 32 rows and two k-blocks a
  // wavefront (one x 7168 x 2048) 10.9 : 12.1.
  auto direct = [&]() { return rows <= kThin8Direct || per <= kThin8Run / 2; };
  auto tokens = [&](int s0) {
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(g.a + (int64_t)row0 * K), (short)0, rows * K, 0x00020000);
    const bool in = direct();
    const int row = in ? r16 : lrow, far = in ? 0 : 8 * K;   // of the two halves of a block
    const unsigned c0 = 16u * (in ? quad : lane & 7), c1 = in ? c0 + 64u : c0;
#pragma unroll
    for (int d = 0; d < kThin8Run; ++d) {
      const int b = s0 + d < per ? kb0 + s0 + d : nk;
      const unsigned k0 = (unsigned)b * kGmm8Block + c0, k1 = (unsigned)b * kGmm8Block + c1;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const unsigned at = (unsigned)((16 * m + row) * K);
        tok[d][m] = join(__builtin_amdgcn_raw_buffer_load_b128(ra, k0 < (unsigned)K ? at + k0 : kPastEnd, 0, 0),
                         __builtin_amdgcn_raw_buffer_load_b128(ra, k1 < (unsigned)K ? at + far + k1 : kPastEnd, 0, 0));
      }
    }
  };
  // through the wavefront's place for the sums of tile t
  auto place = [&](int t) {
    if (direct()) return;
    const unsigned at = sm.red + (t & 1) * (kGmmWaves * MB * 1024) + wave * (MB * 1024);
    const unsigned put = at + lrow * kGmm8Block + (((lane & 7) ^ (lrow >> 1)) << 4), far = at + (8 + lrow) * kGmm8Block +
                                                                                          (((lane & 7) ^ (4 + (lrow >> 1))) << 4);
    const unsigned g0 = at + r16 * kGmm8Block + ((quad ^ key) << 4), g1 = at + r16 * kGmm8Block + (((4 + quad) ^ key) << 4);
#pragma unroll
    for (int d = 0; d < kThin8Run; ++d)
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const v8i q = tok[d][m];
        lds_put(put, __builtin_bit_cast(v4f, v4i{q[0], q[1], q[2], q[3]}));
        lds_put(far, __builtin_bit_cast(v4f, v4i{q[4], q[5], q[6], q[7]}));
        tok[d][m] = lds_get2(g0, g1);   // (a wavefront's LDS accesses keep their order)
      }
  };
  expert();
  tokens(0);
#pragma unroll
  for (int d = 0; d < kSlots; ++d) fetch();

  place(t0);

  const unsigned f0 = sm.ring + r16 * kGmm8Block + ((quad ^ key) << 4);
  const unsigned f1 = sm.ring + r16 * kGmm8Block + (((4 + quad) ^ key) << 4);
  unsigned read = 0;
  for (int t = t0; t < t1; ++t) {
    if (i != have) expert();
    v4i acc[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[m] = v4i{0, 0, 0, 0};
    for (int s0 = 0; s0 < per; s0 += kThin8Run) {
      if (i != have || s0 != held) {
        tokens(s0);
        place(t);
        held = s0;
      }
#pragma unroll
      for (int d = 0; d < kThin8Run; ++d) {
        if (s0 + d < per) {
          __builtin_amdgcn_s_waitcnt(0x0F70 | ((kSlots - 1) * 2));   // at most the loads of the other slots are out
          const v8i w = lds_get2(f0 + read, f1 + read);
          read = read + kSlot == kSlots * kSlot ? 0 : read + kSlot;
          fetch();
          const v4i w0 = {w[0], w[1], w[2], w[3]}, w1 = {w[4], w[5], w[6], w[7]};
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            const v8i q = tok[d][m];
            acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, v4i{q[0], q[1], q[2], q[3]}, acc[m], 0, 0, 0);
            acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, v4i{q[4], q[5], q[6], q[7]}, acc[m], 0, 0, 0);
          }
        }
      }
      have = i;
    }
    // join the runs of k-blocks: job (column block, row block) by another wavefront for each tile
    const unsigned red = sm.red + (t & 1) * (kGmmWaves * MB * 1024);
    matrix_done(acc);
#pragma unroll
    for (int m = 0; m < MB; ++m) lds_put(red + ((wave * MB + m) * 64 + lane) * 16, __builtin_bit_cast(v4f, acc[m]));
    lds_barrier();
    for (int job = (wave + MB * t) & (kGmmWaves - 1); job < MB * rs; job += kGmmWaves) {
      const int ob = job / MB, m = job % MB;
      const int col0 = n0 + 16 * ob;
      if (16 * m < rows && col0 < Nw) {
        v4i sum = {0, 0, 0, 0};
        for (int k = 0; k < ks; ++k) {
          const unsigned at = red + (((ob * ks + k) * MB + m) * 64 + lane) * 16;
          const v8i p = lds_get2(at, at);
#pragma unroll
          for (int r = 0; r < 4; ++r) sum[r] += p[r];
        }
        const int row = 16 * m + r16, col = col0 + 4 * quad;
        // the 16 channels' scales by scalar loads: they pass by the direct loads' count
        const scalar_f* p = (const scalar_f*)(g.w_scale + (int64_t)e * Nw);
        v4f sw;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float a0 = scalar(p[min(col0 + r, Nw - 1)]), a1 = scalar(p[min(col0 + 4 + r, Nw - 1)]);
          const float a2 = scalar(p[min(col0 + 8 + r, Nw - 1)]), a3 = scalar(p[min(col0 + 12 + r, Nw - 1)]);
          sw[r] = quad < 2 ? (quad == 0 ? a0 : a1) : (quad == 2 ? a2 : a3);
        }
        if (row < rows && col < Nw) gmm8_store(g, (int64_t)(row0 + row) * Nw + col, gmm8_scale(sum, m == 0 ? sa[0] : sa[1], sw));
      }
    }
    n0 += width;
    if (n0 >= Nw) {
      n0 = 0;
      ++i;
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // no direct load into LDS is left in flight
}

// ks: at least 6 k-blocks per wavefront, and as many tiles as workgroups.
__device__ __forceinline__ int thin8_split(const Gmm8& g, int experts) {
  int ks = g.nk >= 48 ? 8 : g.nk >= 24 ? 4 : g.nk >= 12 ? 2 : 1;
  while (ks < kGmmWaves && experts * ((g.Nw + 128 / ks - 1) / (128 / ks)) < (int)gridDim.x) ks *= 2;
  return ks;
}

// ---------------------------------------------------------------------------
// Experts with more rows: tiles of BM = 32 to 256 rows x 256 weight rows, one
// workgroup per CU walking tiles.  Each k-block of 128 is one stage, loaded global ->
// LDS directly into a ring of S stages while earlier ones are multiplied.  Wavefront
// (wt, wn) holds the token blocks i WT + wt (32 rows each, so that a short tile's
// blocks are shared) x WB weight blocks of 32.
//
// A stage is four steps of 32 k.  The fragments of a step are read while the one
// before it is multiplied; the last step's products run behind the barrier that
// opens the next stage, beside that stage's first reads.
//
// LDS: chunk c (16 bytes) of row r sits at chunk c ^ ((r / 2) & 7) of the row's
// 128 bytes, so that 16 rows read at one chunk cover all banks.
// ---------------------------------------------------------------------------
constexpr int kWide8 = 256;   // weight rows of a tile
constexpr int wide8_stage(int BM) { return (BM + kWide8) * kGmm8Block; }

template <int BM>
struct Wide8 {
  static constexpr int W = kGmmWaves, WT = BM >= 64 ? 2 : 1;   // wavefronts, along the rows
  static constexpr int TB = BM / 32 / WT, WW = W / WT, WB = kWide8 / 32 / WW;
};

template <int BM, int S, int NB>
__device__ __forceinline__ void wide8_kloop(const Gmm8& g, const WideTile& t, unsigned lds,
                                            v16i (&acc)[Wide8<BM>::TB][Wide8<BM>::WB]) {
  typedef Wide8<BM> C;
  constexpr int W = C::W;
  constexpr int kStage = wide8_stage(BM), kRing = S * kStage, kTokenBytes = BM * kGmm8Block;
  constexpr int kWeightLoads = 32 / W, kTokenLoads = BM / 8 >= W ? BM / 8 / W : 1;
  constexpr int kLoads = kWeightLoads + kTokenLoads, kParts = S == 2 ? 2 : 4, kPart = (kLoads + kParts - 1) / kParts;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wt = wave / C::WW, wn = wave % C::WW;
  const int K = g.K, nk = g.nk, Nw = g.Nw;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(g.a + (int64_t)t.row0 * K), (short)0, t.rows * K, 0x00020000);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(g.w + ((int64_t)t.e * Nw + t.n0) * K), (short)0, (Nw - t.n0) * K, 0x00020000);
  unsigned vo[2], chunk[2];   // lane part of a load of eight rows, by the parity of its place
#pragma unroll
  for (int par = 0; par < 2; ++par) {
    chunk[par] = (unsigned)(((lane & 7) ^ ((4 * par + (lane >> 4)) & 7)) << 4);
    vo[par] = (unsigned)((lane >> 3) * K) + chunk[par];
  }
  // direct loads of k-block b into the stage at `at` of the ring, in four parts
  auto dma = [&](int at, int b, int part) {
    unsigned v[2];
    const unsigned k0 = (unsigned)b * kGmm8Block;
#pragma unroll
    for (int par = 0; par < 2; ++par) v[par] = k0 + chunk[par] < (unsigned)K ? vo[par] : kPastEnd;   // zeros past K
    // (offsets step by step: hoisted out of the loop they would take a scalar register each)
    unsigned so = k0 + (unsigned)(8 * kWeightLoads * K) * (unsigned)wave, st = k0 + (unsigned)(8 * kTokenLoads * K) * (unsigned)wave;
#pragma unroll
    for (int q = part * kPart; q < min(kLoads, (part + 1) * kPart); ++q) {
      if (q == part * kPart && q < kWeightLoads) so += (unsigned)(8 * q * K);
      if (q == part * kPart && q > kWeightLoads) st += (unsigned)(8 * (q - kWeightLoads) * K);
      if (q < kWeightLoads) {
        asm("" : "+s"(so));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(size_t)(lds + at + kTokenBytes + (kWeightLoads * wave + q) * 1024), 16,
                                                 v[q & 1], so, 0, 0);
        so += 8u * (unsigned)K;
      } else {
        asm("" : "+s"(st));
        const int blk = (kTokenLoads * wave + q - kWeightLoads) & (BM / 8 - 1);   // (BM = 32, W = 8: two load the same)
        const unsigned off = BM / 8 >= W ? st : k0 + (unsigned)(8 * blk * K);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(size_t)(lds + at + blk * 1024), 16, v[blk & 1], off, 0, 0);
        st += 8u * (unsigned)K;
      }
    }
  };
  // fragments: lane l reads row l % 32 of a block, chunk 2 q + l / 32 of step q
  typedef const __attribute__((address_space(3))) v4i lds_v4i;
  unsigned fr[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    fr[q] = lds + (lane & 31) * kGmm8Block + (((2 * q + (lane >> 5)) ^ ((lane >> 1) & 7)) << 4);
  v4i tf[2][NB], wf[2][C::WB];
  auto frags = [&](int at, int q) {
#pragma unroll
    for (int i = 0; i < NB; ++i) tf[q & 1][i] = *(lds_v4i*)(size_t)(fr[q] + at + 32 * (i * C::WT + wt) * kGmm8Block);
#pragma unroll
    for (int j = 0; j < C::WB; ++j)
      wf[q & 1][j] = *(lds_v4i*)(size_t)(fr[q] + at + kTokenBytes + 32 * (wn * C::WB + j) * kGmm8Block);
  };
  auto mfmas = [&](int q) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < C::WB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[q & 1][j], tf[q & 1][i], acc[i][j], 0, 0, 0);
  };
  constexpr int NR = NB + C::WB, NM = NB * C::WB;
  // the step's reads and direct loads between its products
  auto interleave = [&](bool loads) {
#pragma unroll
    for (int n = 0; n < (NR > NM ? NR : NM); ++n) {
      if (n < NM) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (n < NR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (loads && n < kPart) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int kAhead = 0x0F70 | (((S - 2) * kLoads) & 15) | ((((S - 2) * kLoads) >> 4) << 14);   // vmcnt of S - 2 stages
#pragma unroll
  for (int d = 0; d < S - 1; ++d)
#pragma unroll
    for (int part = 0; part < kParts; ++part) dma(d * kStage, d, part);
  __builtin_amdgcn_s_waitcnt(kAhead);   // this wavefront's loads of stage 0 have landed
  lds_barrier();
  dma((S - 1) * kStage, S - 1, 0);
  frags(0, 0);
  int cur = 0, nxt = kStage, last = (S - 1) * kStage;   // places of k-blocks b, b + 1, b + S - 1
  for (int b = 0; b < nk; ++b) {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      frags(cur, q + 1);
      if (q + 1 < kParts) dma(last, b + S - 1, q + 1);
      mfmas(q);
      interleave(q + 1 < kParts);
    }
    __builtin_amdgcn_s_waitcnt(kAhead);   // this wavefront's loads of k-block b + 1 have landed
    lds_barrier();
    frags(nxt, 0);   // (after the last stage: read, never used)
    dma(cur, b + S, 0);
    mfmas(3);
    interleave(true);
    last = cur;
    cur = nxt;
    nxt = nxt + kStage == kRing ? 0 : nxt + kStage;
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): the loads past the last stage (of zeros) have landed too
}

// One tile: the k loop, then the outputs, 16-bit ones through LDS as whole rows.
template <int BM, int S>
__device__ __forceinline__ void wide8_tile(const Gmm8& g, const WideTile& t, uint8_t* smem) {
  typedef Wide8<BM> C;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / C::WW, wn = wave % C::WW;
  v16i acc[C::TB][C::WB];
#pragma unroll
  for (int i = 0; i < C::TB; ++i)
#pragma unroll
    for (int j = 0; j < C::WB; ++j) acc[i][j] = v16i{};
  const unsigned lds = lds_at(smem);
  const int blocks = (t.rows + 32 * C::WT - 1) / (32 * C::WT);   // of each wavefront that hold rows
  if constexpr (C::TB == 1) wide8_kloop<BM, S, 1>(g, t, lds, acc);
  else if constexpr (C::TB == 2) {
    if (blocks > 1) wide8_kloop<BM, S, 2>(g, t, lds, acc);
    else wide8_kloop<BM, S, 1>(g, t, lds, acc);
  } else {
    if (blocks > 3) wide8_kloop<BM, S, 4>(g, t, lds, acc);
    else if (blocks > 2) wide8_kloop<BM, S, 3>(g, t, lds, acc);
    else if (blocks > 1) wide8_kloop<BM, S, 2>(g, t, lds, acc);
    else wide8_kloop<BM, S, 1>(g, t, lds, acc);
  }
  const __amdgpu_buffer_rsrc_t rc = channel_scales(g, t.e);
  v4f sw[C::WB][4];
  float sa[C::TB];
#pragma unroll
  for (int j = 0; j < C::WB; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      sw[j][q] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(
                                             rc, (unsigned)(t.n0 + 32 * (wn * C::WB + j) + 8 * q + 4 * (lane >> 5)) * 4u, 0, 0));
#pragma unroll
  for (int i = 0; i < C::TB; ++i) sa[i] = g.a_scale[t.row0 + min(32 * (i * C::WT + wt) + (lane & 31), t.rows - 1)];
  __syncthreads();   // every wavefront has left the ring
  auto outputs = [&](auto&& put) {   // put(row, column, four values): those of the tile
#pragma unroll
    for (int i = 0; i < C::TB; ++i)
#pragma unroll
      for (int j = 0; j < C::WB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          put(32 * (i * C::WT + wt) + (lane & 31), 32 * (wn * C::WB + j) + 8 * q + 4 * (lane >> 5),
              gmm8_scale(v4i{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]}, sa[i], sw[j][q]));
  };
  const bool wide = g.dtype == MDC_DTYPE_FP32;
  auto place = [&](int row, int in) {   // 16-byte units of 8 columns
    return smem + row * 512 + (((in >> 3) ^ (row & 31)) << 4) + 8 * (lane >> 5);
  };
  if (wide)
    outputs([&](int row, int in, v4f v) {
      if (row < t.rows && t.n0 + in < g.Nw)
        *reinterpret_cast<v4f*>(static_cast<float*>(g.y) + (int64_t)(t.row0 + row) * g.Nw + t.n0 + in) = v;
    });
  else if (g.dtype == MDC_DTYPE_BF16)
    outputs([&](int row, int in, v4f v) { *reinterpret_cast<v4b*>(place(row, in)) = __builtin_convertvector(v, v4b); });
  else outputs([&](int row, int in, v4f v) { *reinterpret_cast<v4h*>(place(row, in)) = __builtin_convertvector(v, v4h); });
  if (!wide) {
    __syncthreads();
    const int unit = tid & 31, col = t.n0 + 8 * unit;
    if (col < g.Nw)
      for (int r = tid >> 5; r < t.rows; r += kGmmThreads / 32)
        __builtin_nontemporal_store(*reinterpret_cast<const v4u*>(smem + r * 512 + ((unit ^ (r & 31)) << 4)),
            reinterpret_cast<v4u*>(static_cast<uint16_t*>(g.y) + (int64_t)(t.row0 + r) * g.Nw + col));
  }
  lds_barrier();   // the ring is free
}

template <int BM, int S>
__device__ __forceinline__ void wide8_walk(const Gmm8& g, const GmmTable& tab, uint8_t* smem) {
  const int nn = (g.Nw + kWide8 - 1) / kWide8;
  const int T = tab.tiles[g.L] * nn;
  for (int t = wide_line(); t < T; t += gridDim.x) wide8_tile<BM, S>(g, wide_place(g, tab, t, nn, BM, kWide8), smem);
}

// ---------------------------------------------------------------------------
// Experts of more rows in a call of few tiles: tiles of 64 rows x 64 weight rows,
// whose k-blocks go round the eight wavefronts.  A wavefront has the whole tile's
// sums, 64 registers, and a k-block of its own in LDS, 128 bytes of each row: no
// barrier until the eight sums are joined.  What bounds it is the 16 KB a k-block
// from the caches, twice what a tile of 256 x 256 takes for a product, and the time
// until they come; for one round of tiles it is the shorter way.  64 rows of one
// expert x 4096 x 7168: 22.8 us, with tiles of 32 x 256 43; 500 x 1160 x 2000 9.6
// and 15.8; 64 of each of four x 4096 x 7168 27.8 and 48.5.  (By 64 bytes of each
// row at a time, in two slots, 32; straight from memory into registers, where lanes
// side by side read different rows, 32.)
// ---------------------------------------------------------------------------
constexpr int kSplit8 = 64;   // rows and weight rows of a tile

__device__ __forceinline__ void split8_walk(const Gmm8& g, const GmmTable& tab, uint8_t* smem) {
  constexpr int B = kSplit8 / 16, kSlot = 2 * kSplit8 * kGmm8Block;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const int K = g.K, Nw = g.Nw;
  const int nn = (Nw + kSplit8 - 1) / kSplit8;
  const int T = tab.tiles[g.L] * nn;
  const int steps = (g.nk + kGmmWaves - 1) / kGmmWaves;   // k-blocks of a wavefront
  const unsigned lds = lds_at(smem), ring = lds + wave * kSlot;
  const int lrow = lane >> 3, key = (r16 >> 1) & 7;
  const unsigned f0 = ring + r16 * kGmm8Block + ((quad ^ key) << 4), f1 = ring + r16 * kGmm8Block + (((4 + quad) ^ key) << 4);
  __amdgpu_buffer_rsrc_t ra, rw;
  auto fetch = [&](int step) {
    const unsigned k0 = (unsigned)(kGmmWaves * step + wave) * kGmm8Block;
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // eight rows each, as a thin expert's weights
      const unsigned chunk = (unsigned)((lane & 7) ^ ((4 * h + (lrow >> 1)) & 7)) << 4;
      const unsigned v = k0 + chunk < (unsigned)K ? (unsigned)((8 * h + lrow) * K) + k0 + chunk : kPastEnd;   // zeros past K
#pragma unroll
      for (int m = 0; m < B; ++m) {
        const unsigned rows = (unsigned)(16 * m * K);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(size_t)(ring + (2 * m + h) * 1024), 16, v + rows, 0, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(size_t)(ring + (2 * (B + m) + h) * 1024), 16, v + rows, 0, 0, 0);
      }
    }
  };
  typedef const __attribute__((address_space(3))) v4i lds_v4i;
  for (int t = wide_line(); t < T; t += gridDim.x) {
    const WideTile tile = wide_place(g, tab, t, nn, kSplit8, kSplit8);
    ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(g.a + (int64_t)tile.row0 * K), (short)0, tile.rows * K, 0x00020000);
    rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(g.w + ((int64_t)tile.e * Nw + tile.n0) * K), (short)0,
                                           (Nw - tile.n0) * K, 0x00020000);
    // blocks (m, c) and (m, c + 1) of 16 x 16 are this wavefront's to store
    const int m = wave / 2, c = wave % 2 * 2, row = 16 * m + r16;
    const __amdgpu_buffer_rsrc_t rc = channel_scales(g, tile.e);
    v4f sw[2];
    const float sa = g.a_scale[tile.row0 + min(row, tile.rows - 1)];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      sw[j] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rc, (unsigned)(tile.n0 + 16 * (c + j) + 4 * quad) * 4u, 0, 0));
    v4i acc[B][B];
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int j = 0; j < B; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    fetch(0);
    for (int s = 0; s < steps; ++s) {
      v4i q[2][B], w[2][B];
      __builtin_amdgcn_s_waitcnt(0x0F70);   // the k-block is there
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < B; ++i) {
          q[h][i] = *(lds_v4i*)(size_t)((h == 0 ? f0 : f1) + i * 2048);
          w[h][i] = *(lds_v4i*)(size_t)((h == 0 ? f0 : f1) + (B + i) * 2048);
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // it has been read
      __builtin_amdgcn_sched_barrier(0);
      fetch(s + 1);   // (past the last: zeros, never used)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
          for (int j = 0; j < B; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][j], q[h][i], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);   // no direct load into LDS is left in flight
    lds_barrier();                        // the rings are free
    matrix_done(acc);
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int j = 0; j < B; ++j) lds_put(lds + (((wave * B + i) * B + j) * 64 + lane) * 16, __builtin_bit_cast(v4f, acc[i][j]));
    lds_barrier();
    if (row - r16 < tile.rows) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v4i sum = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kGmmWaves; k += 2) {
          const unsigned at = lds + (((k * B + m) * B + c + j) * 64 + lane) * 16;
          const v8i p = lds_get2(at, at + B * B * 1024);
#pragma unroll
          for (int r = 0; r < 4; ++r) sum[r] += p[r] + p[4 + r];
        }
        const int col = tile.n0 + 16 * (c + j) + 4 * quad;
        if (row < tile.rows && col < Nw) gmm8_store(g, (int64_t)(tile.row0 + row) * Nw + col, gmm8_scale(sum, sa, sw[j]));
      }
    }
    lds_barrier();   // the sums have been read
  }
}

// What a k-block of a tile of 256, 128, 64 and 32 rows takes, and one of a tile whose
// k-blocks are split, in hundredths of a microsecond; there the join's time too.
// (Rounds of 56 k-blocks of the split tiles: 15.4 us; of 16: 6.)
constexpr int kCost8[4] = {200, 120, 80, 60}, kCost8_Split = 24, kCost8_Join = 200;

// LDS of the tiles; 128-row tiles take three stages and 32-row tiles four where the experts' table leaves that much.
constexpr int kLds8Deep = 3 * wide8_stage(128), kLds8Flat = 2 * wide8_stage(256);
static_assert(kLds8Flat >= 3 * wide8_stage(64) && kLds8Flat >= 3 * wide8_stage(32) && kLds8Deep >= 4 * wide8_stage(32) &&
                  kLds8Deep >= kLds8Flat && kLds8Flat >= kGmmWaves * kThin8Ring + 2 * kGmmWaves * kThinBlocks * 1024 &&
                  kLds8Flat >= kGmmWaves * kSplit8 * kSplit8 * 4,   // (the rings are as large)
              "LDS of the tiles");

// How the experts of more than kThinRows rows are cut: tiles of `rows` rows, the
// k-blocks of a tile one after another or over the wavefronts (split).
struct Wide8Plan {
  int rows = 0;   // 0: there are no such experts
  bool split = false;
  int tiles = 0;
  __device__ int cost() const { return split ? 2 : 16; }   // of a tile, in those of 16 columns of thin work
};

// count: m-tiles of 256, 128, 64 and 32 rows.
__device__ __forceinline__ Wide8Plan wide8_plan(const Gmm8& g, const int (&count)[4]) {
  // Tiles of 256, 128, 64 or 32 rows, whichever rounds of tiles take less time:
  // large ones do more products per byte and stage, small ones fill the CUs.
  const int G = gridDim.x, nn = (g.Nw + kWide8 - 1) / kWide8;
  Wide8Plan p;
  int64_t least = INT64_MAX;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t c = (int64_t)kCost8[i] * ((count[i] * nn + G - 1) / G) * g.nk;
    if (c < least) {
      p.rows = 256 >> i;
      p.tiles = count[i] * nn;
      least = c;
    }
  }
  const int tiles = count[2] * ((g.Nw + kSplit8 - 1) / kSplit8);
  const int64_t c = (int64_t)((tiles + G - 1) / G) * (kCost8_Split * g.nk + kCost8_Join);
  if (c < least) {
    p.rows = kSplit8;
    p.tiles = tiles;
    p.split = true;
  }
  return p;
}

// The plan of up to 64 experts, lane e's expert e, by each wavefront for itself:
// no barrier but the one behind it.  (One row of one expert x 7168 x 2048: the whole
// kernel 9.4 us, and 10.8 with the scans of the workgroup; 3001 rows of 6 experts x
// 1160 x 2000 19.1 and 20.4.)
__device__ __forceinline__ Wide8Plan gmm8_few(const Gmm8& g, GmmTable& t) {
  const int lane = threadIdx.x & 63;
  const int64_t v = lane < g.L ? gmm_count(g.nums, lane, g.A) : 0;
  // in two halves of at most 30 bits' sum each
  const int64_t low = wave_inclusive_scan((int)(v & 0xFFFFFF));
  const int end = (int)min(((int64_t)wave_inclusive_scan((int)(v >> 24)) << 24) + low, (int64_t)g.A);
  const int before = __shfl_up(end, 1, 64);   // (by all lanes: of one that is off it would be zero)
  const int n = lane < g.L ? end - (lane == 0 ? 0 : before) : 0;
  const bool thin = n > 0 && n <= kThinRows;
  const uint64_t thins = __ballot(thin);
  t.n_thin = __builtin_amdgcn_readfirstlane(__popcll(thins));
  Wide8Plan p;
  if (__any(n > kThinRows)) {
    int count[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      count[i] = __builtin_amdgcn_readlane(wave_inclusive_scan(n > kThinRows ? (n - 1) / (256 >> i) + 1 : 0), 63);
    p = wide8_plan(g, count);
    const int tiles = wave_inclusive_scan(n > kThinRows ? (n - 1) / p.rows + 1 : 0);
    if (threadIdx.x < g.L) t.tiles[lane + 1] = tiles;
    if (threadIdx.x == 0) t.tiles[0] = 0;
  }
  if (threadIdx.x < g.L) t.rows[lane + 1] = end;
  if (threadIdx.x == 0) t.rows[0] = 0;
  if (threadIdx.x < 64 && thin) t.thin[__popcll(thins & lanes_below(lane))] = (uint16_t)lane;
  __syncthreads();
  return p;
}

// The same of any number of experts.
__device__ __forceinline__ Wide8Plan gmm8_many(const Gmm8& g, GmmTable& t, int64_t* wave_total) {
  gmm_rows<kGmmThreads>(g, t.rows, wave_total);
  int count[4], fewer[3];
  count[0] = gmm_tiles(g, t, 256, wave_total);
  if (count[0] == 0) return Wide8Plan();
  gmm_tile_counts(g, t, fewer);
#pragma unroll
  for (int i = 0; i < 3; ++i) count[i + 1] = fewer[i];
  const Wide8Plan p = wide8_plan(g, count);
  if (p.rows != 256) gmm_tiles(g, t, p.rows, wave_total);
  return p;
}

// One workgroup per CU: the wide experts' tiles, then the thin experts'.  All ways in
// one kernel take 256 registers, and ten more that spill (44 bytes of scratch): they
// come back once a tile around the k loop of the 256-row tiles and in their outputs,
// never inside a loop over k.
template <bool DEEP>
__global__ __launch_bounds__(kGmmThreads) void k_gmm8(Gmm8 g) {
  extern __shared__ int gmm_table[];
  __shared__ __attribute__((aligned(16))) uint8_t smem[DEEP ? kLds8Deep : kLds8Flat];
  __shared__ int64_t wave_total[kGmmWaves];
  GmmTable tab{gmm_table, gmm_table + g.L + 1, reinterpret_cast<uint16_t*>(gmm_table + 2 * (g.L + 1)), 0};
  const Wide8Plan p = g.L <= 64 ? gmm8_few(g, tab) : gmm8_many(g, tab, wave_total);
  if (p.split) split8_walk(g, tab, smem);
  else if (p.rows == 32) wide8_walk<32, DEEP ? 4 : 3>(g, tab, smem);
  else if (p.rows == 64) wide8_walk<64, 3>(g, tab, smem);
  else if (p.rows == 128) wide8_walk<128, DEEP ? 3 : 2>(g, tab, smem);
  else if (p.rows == 256) wide8_walk<256, 2>(g, tab, smem);
  if (tab.n_thin != 0) {
    if (p.rows != 0) __syncthreads();   // smem is free
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    thin8_walk(g, tab, p.tiles, p.cost(), thin8_split(g, tab.n_thin),
               Thin8Smem{lds_at(smem) + wave * kThin8Ring, lds_at(smem) + kGmmWaves * kThin8Ring});
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
void launch_gmm8(const Gmm8& g, hipStream_t s) {
  const dim3 grid((device_cus() + 7) / 8 * 8), block(kGmmThreads);
  const size_t table = gmm_table_bytes(g.L);
  if (table + kLds8Deep + 256 <= kLdsSize)   // (256: the plan's few words)
    hipLaunchKernelGGL(k_gmm8<true>, grid, block, table, s, g);
  else hipLaunchKernelGGL(k_gmm8<false>, grid, block, table, s, g);
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
