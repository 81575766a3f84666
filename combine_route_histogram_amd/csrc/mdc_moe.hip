// libmdc: a whole layer of experts for a few tokens, for AMD Instinct MI355X
// (gfx950): mdc_moe (int8 experts), mdc_moe_fp8 (e4m3 experts).

#include "mdc_gate.h"
#include "mdc_group.h"

namespace {

// ---------------------------------------------------------------------------
// x_out[t] = sum over the token's routes of scale * (W2 q(silu(W1g q(x)) * W1u
// q(x)) + shared), all experts of all tokens in three launches:
//
//   k_moe_prep  the gate, and q(x), a workgroup each for a token
//   k_moe_up    h = q(x) W1^T for every expert that has a token, and SwiGLU: g,
//               fp32, into the workspace
//   k_moe_down  q(g) W2^T times the routes' scales, summed over the experts
//
// With at most 32 tokens an expert's rows fill one or two blocks of the matrix
// instruction, and what takes the time is to bring the weights of the experts in
// use, once.  The last two kernels run one workgroup of eight wavefronts per CU, each
// wavefront streaming weights global -> LDS directly through a ring of its own
// (eight rows x 128 bytes per instruction, non-temporal: they are read once).
//
// k_moe_up: a tile is 8 gate columns and the 8 up columns that go with them, one
// 16-row block of the matrix instruction; the wavefronts split k.  Every token is
// an operand row for every expert, so the tokens' codes stay in registers for the
// whole kernel; rows of tokens that an expert does not have are computed and
// dropped.  The sums of the eight wavefronts are joined through LDS, by another
// wavefront for each tile.
//
// k_moe_down: a workgroup has the columns [cw b, cw (b + 1)) of the output and
// walks all experts: no sum leaves the workgroup.  A unit of work is a k-block of
// 128 of one expert; wavefront w takes units w, w + 8, ... and keeps sums for all
// tokens in registers, scaled by its rows' route scales as they are added.  The
// rows of g are quantised into LDS by all threads, as many units at a time as it
// holds cells (a cell is 128 values of one row).
//
// Sums are fp32 (int32 inside an int8 product), in an order that depends on the
// routes only.  g stays fp32 until it is quantised: a block of it (int8: a row) is
// the work of several workgroups of k_moe_up, so that its scale is known in
// k_moe_down first, which quantises it for each workgroup anew.
//
// Bound: the weights' way from memory, and what stands before it in each launch.
// 8 experts of fp8, 7168 x 4096, one token: 4.8 + 38.7 + 23.3 us, the products at
// 6.1 and 5.0 TB/s, where such loads alone reach 6.8; 13 of them for 32 tokens 5.0 +
// 63 + 42.6; 12 of int8 for 16 tokens 4.7 + 55.5 + 38; 32 of int8, 2048 x 1536, for
// 5 tokens 4 + 22 + 21.4 (1536 columns: 22 us of weights in all); 4 of 1024 x 1024,
// one token 2.6 + 6.6 + 7.6.  Before its first product k_moe_up takes 4 us (routes,
// table, the tokens' codes), k_moe_down 5 to 7 (the table, g and its quantisation),
// by clocks read in the kernel; weights are on their way for half of that.  Held
// against it: the tokens quantised inside k_moe_up (spills; one token 98 us, 85 with
// k_moe_prep), the rows' largest values by atomics instead of one for each tile (8 us
// more at 16 tokens, all workgroups meet at few words).
// ---------------------------------------------------------------------------
constexpr int kMoeThreads = 512;
constexpr int kMoeWaves = kMoeThreads / 64;
constexpr int kMoeTokens = MDC_MAX_MOE_TOKENS;
constexpr int kMoeRoutes = kMoeTokens * MDC_MAX_TOPK;
constexpr int kMoeNt = 2;             // cache policy of the weights' loads: non-temporal
constexpr int kUpRing = 12288;        // bytes of a wavefront's ring
constexpr int kDownRing = 12288;
constexpr int kUpRun = 8;             // most k-blocks of a wavefront
constexpr int kCells = 256;           // rows x k-blocks of g in LDS at a time
constexpr int kTops = 8;              // int8: largest values of tiles in a thread's registers
constexpr int kGroupExperts = 64;     // int8: and experts' channel scales
static_assert(kMoeRoutes <= kMoeThreads, "a thread for each route");

struct MoeTable;
struct Moe {
  const void* x;             // [T][H] bf16
  uint8_t* q;                // codes of x as k_moe_up loads them: moe_code
  float* q_scale;            // int8: [T]; fp8: [H / 128][kMoeTokens]
  MoeTable* table;           // as k_moe_up worked it out, for k_moe_down
  const int32_t* ids;        // [T][K]
  const float* scales;       // [T][K]
  const uint8_t* mask;       // [T] or [T][K], or NULL
  const uint8_t* w1;         // [L][N][H]
  const float* w1_scale;     // int8: [L][N]; fp8: [L][N / 128][H / 128]
  const uint8_t* w2;         // [L][H][N / 2]
  const float* w2_scale;     // int8: [L][H]; fp8: [L][H / 128][N / 256]
  const uint16_t* shared;    // [T][H] bf16, or NULL
  const uint16_t* ori;       // [T][H] bf16, or NULL
  uint16_t* out;             // [T][H] bf16
  float* g;                  // [rows N / 256][128]: cells, by expert, k-block and row
  float* g_max;              // int8: [rows][N / 16] largest |g| of each tile
  mdc_device_status* status;
  int T, K, H, N, L;
  int first;                 // id of local expert 0
  int E, EZ, all;            // ids: routed, routed and zero, all of them
  int per_route;
  int cw;                    // output columns of a workgroup
};

// ---------------------------------------------------------------------------
// The routes as both kernels see them: the experts in use, in the order of their
// first routes, with the tokens that they have.
// ---------------------------------------------------------------------------
struct MoeTable {
  uint16_t expert[kMoeRoutes];
  uint32_t tokens[kMoeRoutes];      // bit t: token t has a route to it
  int base[kMoeRoutes + 1];         // rows of the experts before it
  float weight[kMoeRoutes];         // of each row: the sum of its routes' scales
  float copy[kMoeTokens];           // sum of the scales of the token's copy experts
  float present[kMoeTokens];        // and of all its routes
  uint32_t has[kMoeTokens];         // bit 0: it has a route to a copy expert; bit 1: a present route
  int wave_total[kMoeWaves];
  int experts, dropped;
};

// By all threads of a workgroup, the entries of R routes; no barrier.
__device__ __forceinline__ void table_copy(MoeTable& to, const MoeTable& from, int R) {
  const int i = threadIdx.x;
  if (i < R) {
    const uint16_t e = from.expert[i];
    const uint32_t t = from.tokens[i];
    const int b = from.base[i + 1];
    const float w = from.weight[i];
    to.expert[i] = e;
    to.tokens[i] = t;
    to.base[i + 1] = b;
    to.weight[i] = w;
  }
  if (i < kMoeTokens) {
    const float c = from.copy[i], p = from.present[i];
    const uint32_t h = from.has[i];
    to.copy[i] = c;
    to.present[i] = p;
    to.has[i] = h;
  }
  if (i == 0) {
    to.base[0] = 0;
    to.experts = from.experts;
  }
}

// One route, of thread i; not live: masked, or past the last.
struct MoeRoute {
  int id;
  float scale;
  bool live;
};
__device__ __forceinline__ MoeRoute moe_route(const Moe& a) {
  const int i = threadIdx.x;
  MoeRoute r = {-1, 0.f, false};
  if (i < a.T * a.K) {
    r.id = a.ids[i];
    r.scale = a.scales[i];
    r.live = a.mask == nullptr || a.mask[a.per_route ? i : i / a.K] != 0;
  }
  return r;
}

// Inclusive sum over the workgroup's threads, and the sum of all of them.
__device__ __forceinline__ int moe_scan(int v, int* wave_total, int& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  v = wave_inclusive_scan(v);
  if (lane == 63) wave_total[wave] = v;
  lds_barrier();
  all = 0;
#pragma unroll
  for (int w = 0; w < kMoeWaves; ++w) {
    const int n = wave_total[w];
    if (w < wave) v += n;
    all += n;
  }
  lds_barrier();
  return v;
}

// Threads meet at LDS only: loads that were issued before stay on their way.
// tmp: L ints of LDS, free again afterwards.
__device__ __forceinline__ void moe_table(const Moe& a, const MoeRoute& route, MoeTable& t, int* tmp) {
  __shared__ int ids[kMoeRoutes];        // -1: not present
  __shared__ float scales[kMoeRoutes];
  const int i = threadIdx.x, R = a.T * a.K;
  const int token = i / a.K;
  const int id = route.id;
  const float scale = route.scale;
  const bool live = route.live;
  const bool present = live && id >= 0 && id < a.all;
  const int e = id - a.first;
  const bool mine = present && id < a.E && e >= 0 && e < a.L;
  for (int k = i; k < a.L; k += kMoeThreads) tmp[k] = INT32_MAX;
  if (i == 0) t.dropped = 0;
  t.tokens[i] = 0;
  ids[i] = present ? id : -1;
  scales[i] = scale;
  lds_barrier();
  if (mine) atomicMin(&tmp[e], i);
  if (live && !present) atomicAdd(&t.dropped, 1);
  lds_barrier();
  // place of the expert of each first route
  const bool first = mine && tmp[e] == i;
  int n, rows;
  const int place = moe_scan(first ? 1 : 0, t.wave_total, n) - 1;
  if (first) {
    t.expert[place] = (uint16_t)e;
    tmp[e] = -1 - place;
  }
  if (i == 0) t.experts = n;
  lds_barrier();
  const int j = mine ? -1 - tmp[e] : 0;
  if (mine) atomicOr(&t.tokens[j], 1u << token);
  lds_barrier();
  const int end = moe_scan(__popc(t.tokens[i]), t.wave_total, rows);
  t.base[i + 1] = end;
  if (i == 0) t.base[0] = 0;
  lds_barrier();
  // sums over a token's routes, in order: by the first route of an expert, and by the first of the token
  // (for k_moe_down: only workgroup 0 hands the table on)
  if (blockIdx.x != 0) return;
  if (i < R) {
    float sum = 0.f, copy = 0.f, all = 0.f;
    uint32_t has = 0;
    bool lead = mine;
    const int r0 = token * a.K;
#pragma unroll 4
    for (int r = r0; r < r0 + a.K; ++r) {
      const int other = ids[r];
      const float s = other >= 0 ? scales[r] : 0.f;
      const bool same = other >= 0 && other == id;
      sum += same ? s : 0.f;
      lead = lead && !(same && r < i);
      copy += other >= a.EZ ? s : 0.f;
      all += s;
      has |= (other >= a.EZ ? 1u : 0u) | (other >= 0 ? 2u : 0u);
    }
    if (lead) t.weight[t.base[j] + __popc(t.tokens[j] & ((1u << token) - 1))] = sum;
    if (i == r0) {
      t.copy[token] = copy;
      t.present[token] = all;
      t.has[token] = has;
    }
  }
  lds_barrier();
}

// ---- one product of 16 weight rows x 128 k x 16 tokens ----
// int8: exact.  fp8: the instruction cuts each product of eight consecutive k 2^13
// below the power of two under the largest of them and adds exactly from there (as in
// all fp8 products here; the instruction has no other way).  One token of 8 fp8
// experts is 0.0018-0.0019 from 64 bits (relative L2), plain fp32 products 0.0017:
// bf16's rounding, and codes of g that the cut or silu puts past a border.
template <bool INT8>
struct MoeAcc {
  typedef v4f type;
};
template <>
struct MoeAcc<true> {
  typedef v4i type;
};
__device__ __forceinline__ v4f moe_mfma_fp8(v8i w, v8i t) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, t, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v4i moe_mfma_int8(v8i w, v8i t, v4i c) {
  c = __builtin_amdgcn_mfma_i32_16x16x64_i8(v4i{w[0], w[1], w[2], w[3]}, v4i{t[0], t[1], t[2], t[3]}, c, 0, 0, 0);
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(v4i{w[4], w[5], w[6], w[7]}, v4i{t[4], t[5], t[6], t[7]}, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t int8_codes4(float a, float b, float c, float d, float inv) {
  auto code = [&](float v) { return (uint32_t)(uint8_t)(int8_t)(int)fminf(fmaxf(rintf(v * inv), -127.f), 127.f); };
  return code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
}
__device__ __forceinline__ float int8_inverse(float amax) {
  const float inv = amax > 0.f ? 127.0f / amax : 0.f;
  return inv > 3.402823466e38f ? 3.402823466e38f : inv;
}

// Loads of eight weight rows x 128 bytes into LDS: lane l takes the chunk that
// belongs in slot l % 8 of row l / 8; `odd`: rows 8 .. 15 of the block.
__device__ __forceinline__ unsigned moe_chunk(int lane, int odd) {
  return (unsigned)((lane & 7) ^ ((4 * odd + (lane >> 4)) & 7)) << 4;
}

// ---------------------------------------------------------------------------
// Workgroup (t, 0) quantises token t, workgroup (t, 1) routes it.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;

// Place of chunk c (16 codes) of a token's k-block: k-block, token block, half of
// the chunks, then lane 16 (c % 4) + token % 16 of the matrix instruction, so that
// a load of a fragment is a kilobyte at once.
__device__ __forceinline__ int moe_code(int blocks, int kb, int token, int c) {
  return ((kb * blocks + (token >> 4)) * 2 + (c >> 2)) * 1024 + ((c & 3) * 16 + (token & 15)) * 16;
}

template <typename T, int VPL>
__global__ __launch_bounds__(kPrepThreads) void k_moe_prep(Moe a, GateArgs gate, int int8) {
  extern __shared__ int64_t gate_lds[];
  __shared__ uint32_t part[kPrepThreads / 64];
  const int tid = threadIdx.x, token = blockIdx.x;
  if (blockIdx.y == 1) {
    if (tid < 64) gate_token<T, 64, VPL>(gate, token, true, tid, gate_lds);
    return;
  }
  const int nvec = a.H / 8;   // a multiple of 16, at most 4 a thread
  const v4u* row = static_cast<const v4u*>(a.x) + (int64_t)token * nvec;
  const int blocks = a.T <= 16 ? 1 : 2;
  v4u v[4];
  uint32_t top[4], all = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) v[u] = tid + u * kPrepThreads < nvec ? row[tid + u * kPrepThreads] : v4u{0u, 0u, 0u, 0u};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    top[u] = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) top[u] = max(top[u], max(abs_bits(bf16_lo(v[u][w])), abs_bits(bf16_hi(v[u][w]))));
    top[u] = row16_max(top[u]);
    all = max(all, top[u]);
  }
  float inv = 0.f;
  if (int8) {
#pragma unroll
    for (int o = 32; o >= 16; o >>= 1) all = max(all, (uint32_t)__shfl_xor((int)all, o, 64));
    if ((tid & 63) == 0) part[tid >> 6] = all;
    __syncthreads();
    all = max(max(part[0], part[1]), max(part[2], part[3]));
    inv = int8_inverse(__uint_as_float(all));
    if (tid == 0) a.q_scale[token] = __uint_as_float(all) / 127.0f;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = tid + u * kPrepThreads;
    const v4u w = v[u];
    uint2* q = reinterpret_cast<uint2*>(a.q + moe_code(blocks, i >> 4, token, (i & 15) >> 1) + 8 * (i & 1));
    if (int8) {
      if (i < nvec)
        *q = uint2{int8_codes4(bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1]), inv),
                   int8_codes4(bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3]), inv)};
    } else if (i < nvec) {
      const Fp8Scaler s(top[u]);
      *q = uint2{s.codes4(bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])),
                 s.codes4(bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3]))};
      if ((i & 15) == 0) a.q_scale[(i >> 4) * kMoeTokens + token] = s.scale;
    }
  }
}

// ---------------------------------------------------------------------------
template <bool INT8, int TB>
__global__ __launch_bounds__(kMoeThreads) void k_moe_up(Moe a) {
  typedef typename MoeAcc<INT8>::type Acc;
  __shared__ __attribute__((aligned(16))) uint8_t ring_mem[kMoeWaves * kUpRing];
  __shared__ __attribute__((aligned(16))) v4f red[2][kMoeWaves * TB * 64];
  __shared__ MoeTable tab;
  static_assert(sizeof(ring_mem) >= MDC_MAX_LOCAL_EXPERTS * sizeof(int), "scratch of the table");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const int H = a.H, N = a.N, nk = H / kFp8Block;
  const int kb0 = wave * nk / kMoeWaves, steps = (wave + 1) * nk / kMoeWaves - kb0;   // this wavefront's k-blocks
  const MoeRoute route = moe_route(a);
  // ---- the tokens' codes in the matrix instruction's layout ----
  v8i tok[kUpRun][TB];
  float sa[kUpRun][TB];
  // (no branches here: the waits for the routes count the loads behind them)
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc(a.q + kb0 * TB * 2048, (short)0, steps * TB * 2048, 0x00020000);
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc(a.q_scale + kb0 * kMoeTokens, (short)0, steps * kMoeTokens * 4, 0x00020000);
#pragma unroll
  for (int m = 0; m < TB; ++m) {
    const bool in = 16 * m + r16 < a.T;
    const unsigned at = in ? 16u * lane : kPastEnd, at_scale = in ? 4u * r16 : kPastEnd;
#pragma unroll
    for (int d = 0; d < kUpRun; ++d) {
      tok[d][m] = join(__builtin_amdgcn_raw_buffer_load_b128(rx, at, (d * TB + m) * 2048, 0),
                       __builtin_amdgcn_raw_buffer_load_b128(rx, at, (d * TB + m) * 2048 + 1024, 0));
      sa[d][m] = INT8 ? 0.f
                      : __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, at_scale, (d * kMoeTokens + 16 * m) * 4, 0));
    }
  }
  float row_scale = 0.f;   // int8: of token 16 (lane / 32) + r16
  if (INT8)
    row_scale = a.q_scale[min(16 * (lane >> 5) + r16, a.T - 1)];
  moe_table(a, route, tab, reinterpret_cast<int*>(ring_mem));
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) *a.status = mdc_device_status{tab.dropped, 0, 0, 0};
    table_copy(*a.table, tab, a.T * a.K);
  }
  const int n_exp = __builtin_amdgcn_readfirstlane(tab.experts);
  const int tiles_per = N / 16;
  // this workgroup's tiles: as many as each has, and one more for the first ones
  const int T = n_exp * tiles_per, each = T / (int)gridDim.x, more = T - each * (int)gridDim.x, b = blockIdx.x;
  const int t0 = b * each + min(b, more), t1 = t0 + each + (b < more ? 1 : 0);
  if (t0 == t1) return;

  // ---- weights ----
  constexpr int kSlot = 2048, kSlots = kUpRing / kSlot;
  const unsigned ring = lds_at(ring_mem) + wave * kUpRing;
  auto weights = [&](int j) {
    const int e = __builtin_amdgcn_readfirstlane((int)tab.expert[j]);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.w1 + (int64_t)e * N * H), (short)0, N * H, 0x00020000);
  };
  struct {
    int j, c, step, left;   // expert's place, tile of it, step, tiles to come
  } f = {t0 / tiles_per, t0 % tiles_per, 0, steps > 0 ? t1 - t0 : 0};
  const __amdgpu_buffer_rsrc_t none = __builtin_amdgcn_make_buffer_rsrc(a.q, (short)0, 0, 0x00020000);   // reads as zeros
  __amdgpu_buffer_rsrc_t rw = f.left > 0 ? weights(f.j) : none;
  unsigned slot = 0, so = (unsigned)kb0 * kFp8Block;
  // lane parts of the two loads: rows 8 c + lane / 8 of the gate's and of the up's columns
  unsigned v0 = (unsigned)(8 * f.c + (lane >> 3)) * (unsigned)H + moe_chunk(lane, 0);
  unsigned v1 = (unsigned)(8 * f.c + (lane >> 3) + N / 2) * (unsigned)H + moe_chunk(lane, 1);
  auto fetch = [&]() {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(size_t)(ring + slot), 16, v0, so, 0, kMoeNt);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(size_t)(ring + slot + 1024), 16, v1, so, 0, kMoeNt);
    slot = slot + kSlot == kSlots * kSlot ? 0 : slot + kSlot;
    so += kFp8Block;
    if (++f.step >= steps) {
      f.step = 0;
      so = (unsigned)kb0 * kFp8Block;
      v0 += 8u * (unsigned)H;
      v1 += 8u * (unsigned)H;
      const bool more = --f.left > 0;
      if (++f.c == tiles_per) {
        f.c = 0;
        v0 -= (unsigned)(N / 2) * (unsigned)H;
        v1 -= (unsigned)(N / 2) * (unsigned)H;
        if (more) rw = weights(++f.j);
      }
      if (!more) rw = none;
    }
  };

  // (the table's scratch is free: its last barrier is behind)
#pragma unroll
  for (int d = 0; d < kSlots; ++d) fetch();

  const int key = (r16 >> 1) & 7;
  const unsigned f0 = ring + r16 * kFp8Block + ((quad ^ key) << 4), f1 = ring + r16 * kFp8Block + (((4 + quad) ^ key) << 4);
  unsigned read = 0;
  int j = t0 / tiles_per, c = t0 % tiles_per, e = 0;
  float sc[kUpRun][TB];   // fp8: scales of the tokens times those of the lane's rows, the same for 16 tiles
  for (int t = t0; t < t1; ++t) {
    if (t == t0 || c == 0) e = __builtin_amdgcn_readfirstlane((int)tab.expert[j]);
    if (!INT8 && (t == t0 || c % 16 == 0)) {
      const scalar_f* p = (const scalar_f*)(a.w1_scale + ((int64_t)e * (N / kFp8Block) + c / 16) * nk);
#pragma unroll
      for (int d = 0; d < kUpRun; ++d) {
        const int b = min(kb0 + d, nk - 1);
        const float gate = p[b], up = p[(int64_t)(N / 256) * nk + b];
        const float s = quad < 2 ? gate : up;
#pragma unroll
        for (int m = 0; m < TB; ++m) sc[d][m] = sa[d][m] * s;
      }
    }
    Acc acc[TB];
#pragma unroll
    for (int m = 0; m < TB; ++m) acc[m] = Acc{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < kUpRun; ++d) {
      if (d < steps) {
        __builtin_amdgcn_s_waitcnt(0x0F70 | ((kSlots - 1) * 2));   // at most the loads of the other slots are out
        const v8i w = lds_get2(f0 + read, f1 + read);
        read = read + kSlot == kSlots * kSlot ? 0 : read + kSlot;
        fetch();
        if constexpr (INT8) {
#pragma unroll
          for (int m = 0; m < TB; ++m) acc[m] = moe_mfma_int8(w, tok[d][m], acc[m]);
        } else {
#pragma unroll
          for (int m = 0; m < TB; ++m) {
            const v4f p = moe_mfma_fp8(w, tok[d][m]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[m][r] = __builtin_fmaf(p[r], sc[d][m], acc[m][r]);
          }
        }
      }
    }
    const unsigned buf = lds_at(red[t & 1]);
    if constexpr (INT8) matrix_done(acc);
#pragma unroll
    for (int m = 0; m < TB; ++m) lds_put(buf + ((wave * TB + m) * 64 + lane) * 16, __builtin_bit_cast(v4f, acc[m]));
    lds_barrier();
    // lane (m, half, r16) of one wavefront: token 16 m + r16, four of the tile's columns
    if (wave == (t & (kMoeWaves - 1)) && (TB == 2 || lane < 32)) {
      const int m = lane >> 5, half = quad & 1, token = 16 * m + r16;
      const uint32_t tokens = tab.tokens[j];
      const Acc __attribute__((address_space(3)))* p =
          (const Acc __attribute__((address_space(3)))*)(size_t)(buf + (m * 64 + half * 16 + r16) * 16);
      Acc gate = p[0], up = p[32];
#pragma unroll
      for (int w = 1; w < kMoeWaves; ++w) {
        gate += p[w * TB * 64];
        up += p[w * TB * 64 + 32];
      }
      v4f hg, hu;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        hg[r] = (float)gate[r];
        hu[r] = (float)up[r];
      }
      if constexpr (INT8) {
        // the channels' scales by scalar loads: they pass by the direct loads' count
        const scalar_f* ws = (const scalar_f*)(a.w1_scale + (int64_t)e * N + 8 * c);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float g0 = scalar(ws[r]), g1 = scalar(ws[4 + r]), u0 = scalar(ws[N / 2 + r]), u1 = scalar(ws[N / 2 + 4 + r]);
          hg[r] = hg[r] * row_scale * (half ? g1 : g0);
          hu[r] = hu[r] * row_scale * (half ? u1 : u0);
        }
      }
      if ((tokens >> token) & 1) {
        const int col = 8 * c + 4 * half;
        v4f v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = gmm_silu(hg[r]) * hu[r];
        const int rows = __popc(tokens), row = __popc(tokens & ((1u << token) - 1));
        const int64_t cell = (int64_t)tab.base[j] * (N / 256) + col / kFp8Block * rows + row;
        *reinterpret_cast<v4f*>(a.g + cell * kFp8Block + col % kFp8Block) = v;
        if (INT8) {
          uint32_t top = max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])));
          top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));   // (the other half of the same token)
          if (half == 0) a.g_max[(int64_t)(tab.base[j] + row) * (N / 16) + c] = __uint_as_float(top);
        }
      }
    }
    if (++c == tiles_per) {
      c = 0;
      ++j;
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // no direct load into LDS is left in flight
}

// ---------------------------------------------------------------------------
// LDS by its address as a number, and its stores written out: of an array the
// compiler would think that the direct loads write it, and wait for all of them.
// (A barrier waits for the stores.)
typedef const __attribute__((address_space(3))) v4i lds_v4i;
typedef const __attribute__((address_space(3))) v4f lds_v4f;
typedef const __attribute__((address_space(3))) float lds_float;
typedef const __attribute__((address_space(3))) uint32_t lds_uint;
__device__ __forceinline__ void lds_put32(unsigned at, uint32_t v) { asm volatile("ds_write_b32 %0, %1" ::"v"(at), "v"(v) : "memory"); }
__device__ __forceinline__ void lds_put64(unsigned at, uint2 v) {
  const v2f w = {__uint_as_float(v.x), __uint_as_float(v.y)};
  asm volatile("ds_write_b64 %0, %1" ::"v"(at), "v"(w) : "memory");
}
__device__ __forceinline__ void lds_max32(unsigned at, uint32_t v) { asm volatile("ds_max_u32 %0, %1" ::"v"(at), "v"(v) : "memory"); }

struct MoeGroup {
  int u0, u1, first, used;   // units, first cell, cells
};

// A unit's operands besides the weights.
template <int TB, int NB>
struct MoeUnit {
  v8i tok[TB];
  float s[TB];
  bool has[TB];   // (the others' sums stay: what an expert holds may be infinite or NaN)
  v4f sc[NB];     // int8: scales of the lane's four columns; fp8: [0], of their block of 128
};

// NH: halves of eight columns.
template <bool INT8, int TB, int NH>
__global__ __launch_bounds__(kMoeThreads) void k_moe_down(Moe a) {
  constexpr int NB = (NH + 1) / 2;   // blocks of 16 columns
  __shared__ __attribute__((aligned(16))) uint8_t ring_mem[kMoeWaves * kDownRing];
  __shared__ __attribute__((aligned(16))) uint8_t cells[(kCells + 1) * kFp8Block];   // the last one: zeros
  __shared__ float cell_scale[kCells + 1];   // of its values, times its row's route scale
  __shared__ uint32_t cell_row[kCells];
  __shared__ v4i unit_info[kCells];          // first cell; tokens; place of w2's scales
  // w2's scales: fp8, of the first and of the last column of each block, a unit's; int8, of all columns, an expert's
  __shared__ __attribute__((aligned(16))) float w_scale[INT8 ? kGroupExperts * NB * 16 : kCells * NB * 2];
  __shared__ uint32_t row_top[INT8 ? kMoeRoutes : 1];   // int8: largest |g| of each row
  __shared__ MoeTable tab;
  static_assert(sizeof(ring_mem) >= kMoeWaves * 4 * 64 * 16, "the wavefronts' sums");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const int H = a.H, K2 = a.N / 2, nk = K2 / kFp8Block, R = a.T * a.K;
  const int c0 = blockIdx.x * a.cw, cols = min(a.cw, H - c0);

  const unsigned cell0 = lds_at(cells), scale0 = lds_at(cell_scale), info0 = lds_at(unit_info), w0 = lds_at(w_scale);
  const unsigned row0 = lds_at(cell_row), top0 = lds_at(row_top), weight0 = lds_at(tab.weight);

  // ---- what the units' groups need of memory, in registers ----
  constexpr int kPasses = kCells * 16 / kMoeThreads;   // 16 lanes x 8 values a cell
  constexpr int kScales = (int)(sizeof(w_scale) / sizeof(float)) / kMoeThreads;
  v4f ga[kPasses], gb[kPasses];
  float gs[kScales];
  auto load_cells = [&](int first, int n) {   // n cells, all of which are inside g
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int cell = (tid + p * kMoeThreads) >> 4;
      const v4f* src = reinterpret_cast<const v4f*>(a.g + ((int64_t)first + min(cell, n - 1)) * kFp8Block) + 2 * (tid & 15);
      ga[p] = src[0];
      gb[p] = src[1];
    }
  };
  // (the first cells before it is known how many there are: the workspace has room for every route's)
  load_cells(0, (int)min((int64_t)R * nk, (int64_t)kCells));
  table_copy(tab, *a.table, R);
  // int8: the largest values of the rows' tiles, as many as there are registers for
  const int per = a.N / 16;   // a multiple of 16
  uint32_t tops[INT8 ? kTops : 1];
  if (INT8) {
#pragma unroll
    for (int p = 0; p < kTops; ++p)
      tops[INT8 ? p : 0] = __float_as_uint(a.g_max[min((int64_t)tid + p * kMoeThreads, (int64_t)R * per - 1)]);
    row_top[INT8 ? tid : 0] = 0;
  }
  if (tid < kFp8Block / 4) reinterpret_cast<uint32_t*>(cells + kCells * kFp8Block)[tid] = 0;
  if (tid == 0) cell_scale[kCells] = 0.f;
  __syncthreads();
  const int n_exp = __builtin_amdgcn_readfirstlane(tab.experts);
  const int units = n_exp * nk;

  // ---- weights: units wave, wave + 8, ... ----
  constexpr int kSlot = NH * 1024, kSlots = kDownRing / kSlot;
  const unsigned ring = lds_at(ring_mem) + wave * kDownRing;
  const __amdgpu_buffer_rsrc_t none = __builtin_amdgcn_make_buffer_rsrc(a.q, (short)0, 0, 0x00020000);   // reads as zeros
  __amdgpu_buffer_rsrc_t rw = none;
  int fj = wave / nk, fk = wave - fj * nk;   // expert's place and k-block of the next unit to be loaded
  bool turn = true;                          // another expert than the last one
  unsigned slot = 0, vo[4];   // (NH of them)
#pragma unroll
  for (int h = 0; h < NH; ++h) vo[h] = (unsigned)(8 * h + (lane >> 3)) * (unsigned)K2 + moe_chunk(lane, h & 1);
  auto fetch = [&]() {
    if (turn) {
      rw = none;
      if (fj < n_exp) {
        const int e = __builtin_amdgcn_readfirstlane((int)tab.expert[fj]);
        rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.w2 + ((int64_t)e * H + c0) * K2), (short)0, cols * K2,
                                               0x00020000);
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(size_t)(ring + slot + h * 1024), 16, vo[h],
                                               (unsigned)fk * kFp8Block, 0, kMoeNt);
    slot = slot + kSlot == kSlots * kSlot ? 0 : slot + kSlot;
    fk += kMoeWaves;
    turn = fk >= nk;
    while (fk >= nk) {
      fk -= nk;
      ++fj;
    }
  };
  // ---- groups: as many units as the cells hold rows of ----
  MoeGroup g = {0, 0, 0, 0};
  // (cells before unit u: base[j] nk + (u - j nk) rows of its expert j)
  auto next_group = [&]() {
    g.u0 = g.u1;
    g.first += g.used;
    const int limit = g.first + kCells;
    int whole = 0;   // experts that end inside
    for (int j = lane; j - lane < n_exp; j += 64) whole += __popcll(__ballot(j < n_exp && tab.base[j + 1] * nk <= limit));
    const int base = __builtin_amdgcn_readfirstlane(tab.base[whole]);
    int rows = 0, part = 0;
    if (whole < n_exp) {
      rows = __builtin_amdgcn_readfirstlane(tab.base[whole + 1]) - base;
      part = (limit - base * nk) / rows;
    }
    g.u1 = whole * nk + part;
    g.used = base * nk + part * rows - g.first;
    const int most = (g.u0 / nk + kGroupExperts) * nk;   // whole experts
    if (INT8 && g.u1 > most) {
      g.u1 = most;
      g.used = __builtin_amdgcn_readfirstlane(tab.base[most / nk]) * nk - g.first;
    }
  };
  auto load_scales = [&]() {
    const int j0 = g.u0 / nk;
#pragma unroll
    for (int p = 0; p < kScales; ++p) {
      const int i = tid + p * kMoeThreads;
      int64_t at;
      if (INT8) {
        const int j = min(j0 + i / (16 * NB), (g.u1 - 1) / nk);
        at = (int64_t)tab.expert[j] * H + min(c0 + i % (16 * NB), H - 1);
      } else {
        const int u = min(g.u0 + i / (2 * NB), g.u1 - 1), n = i / 2 % NB, j = u / nk;
        const int col = min(c0 + 16 * n + 15 * (i & 1), H - 1);
        at = ((int64_t)tab.expert[j] * (H / kFp8Block) + col / kFp8Block) * nk + (u - j * nk);
      }
      gs[p] = a.w2_scale[at];
    }
  };
  // the group's units, cells and scales into LDS
  auto place_units = [&]() {
    const int j0 = g.u0 / nk;
    for (int u = g.u0 + tid; u < g.u1; u += kMoeThreads) {
      const int j = u / nk, base = tab.base[j], rows = tab.base[j + 1] - base;
      const int at = base * nk + (u - j * nk) * rows - g.first;
      const v4i info = {at, (int)tab.tokens[j], INT8 ? (j - j0) * NB * 16 : (u - g.u0) * NB * 2, 0};
      lds_put(info0 + (u - g.u0) * 16, __builtin_bit_cast(v4f, info));
      for (int r = 0; r < rows; ++r) lds_put32(row0 + (at + r) * 4, (uint32_t)(base + r));
    }
  };
  auto place_cells = [&]() {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int cell = (tid + p * kMoeThreads) >> 4, u = tid & 15;
      if (cell < g.used) {
        const v4f x = ga[p], y = gb[p];
        const int row = (int)*(lds_uint*)(size_t)(row0 + cell * 4);
        uint2 code;
        float scale;
        if (INT8) {
          const float top = *(lds_float*)(size_t)(top0 + row * 4), inv = int8_inverse(top);
          code = uint2{int8_codes4(x[0], x[1], x[2], x[3], inv), int8_codes4(y[0], y[1], y[2], y[3], inv)};
          scale = top / 127.0f;
        } else {
          uint32_t top = 0;
#pragma unroll
          for (int r = 0; r < 4; ++r) top = max(top, max(abs_bits(x[r]), abs_bits(y[r])));
          const Fp8Scaler s(row16_max(top));
          code = uint2{s.codes4(x[0], x[1], x[2], x[3]), s.codes4(y[0], y[1], y[2], y[3])};
          scale = s.scale;
        }
        if (u == 0) lds_put32(scale0 + cell * 4, __float_as_uint(scale * *(lds_float*)(size_t)(weight0 + row * 4)));
        lds_put64(cell0 + cell * kFp8Block + (((u >> 1) ^ ((cell >> 1) & 7)) << 4) + (u & 1) * 8, code);
      }
    }
  };

  v4f acc[TB][NB];
#pragma unroll
  for (int m = 0; m < TB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = v4f{0.f, 0.f, 0.f, 0.f};
  const int key = (r16 >> 1) & 7;
  const unsigned f0 = ring + r16 * kFp8Block + ((quad ^ key) << 4), f1 = ring + r16 * kFp8Block + (((4 + quad) ^ key) << 4);
  // (the second half of a block that has one half: its first again, whose products nobody looks at)
  const int key8 = ((r16 & 7) >> 1) & 7;
  const unsigned h0 = ring + (r16 & 7) * kFp8Block + ((quad ^ key8) << 4), h1 = ring + (r16 & 7) * kFp8Block + (((4 + quad) ^ key8) << 4);
  auto load_unit = [&](int u, MoeUnit<TB, NB>& x) {
    const v4i info = *(lds_v4i*)(size_t)(info0 + (u - g.u0) * 16);
    const uint32_t tokens = (uint32_t)info[1];
#pragma unroll
    for (int m = 0; m < TB; ++m) {
      const int token = 16 * m + r16;
      x.has[m] = (tokens >> token) & 1;
      const int cell = x.has[m] ? info[0] + __popc(tokens & ((1u << token) - 1)) : kCells, k = (cell >> 1) & 7;
      const unsigned p = cell0 + cell * kFp8Block;
      x.tok[m] = join(*(lds_v4i*)(size_t)(p + ((quad ^ k) << 4)), *(lds_v4i*)(size_t)(p + (((4 + quad) ^ k) << 4)));
      x.s[m] = *(lds_float*)(size_t)(scale0 + cell * 4);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (INT8) {
        x.sc[n] = *(lds_v4f*)(size_t)(w0 + (info[2] + n * 16 + 4 * quad) * 4);
      } else {
        const bool same = (c0 + 16 * n + 4 * quad) / kFp8Block == (c0 + 16 * n) / kFp8Block;
        x.sc[n][0] = *(lds_float*)(size_t)(w0 + (info[2] + n * 2 + (same ? 0 : 1)) * 4);
      }
    }
  };
  unsigned read = 0;
  int mine = wave;   // this wavefront's next unit
  // The first group's scales before the weights: loads come back in their order.
  next_group();
  if (units != 0) load_scales();
#pragma unroll
  for (int d = 0; d < kSlots; ++d) fetch();
  if (INT8) {
    // 16 lanes look at one row (fewer than 2^30 tiles in all)
    const unsigned n = (unsigned)(tab.base[n_exp] * per);
    auto look = [&](unsigned i, uint32_t v) {
      v = row16_max(v);
      if (r16 == 0 && i < n) lds_max32(top0 + i / (unsigned)per * 4, v);
    };
#pragma unroll
    for (int p = 0; p < kTops; ++p)
      if (p * kMoeThreads < n) look(tid + p * kMoeThreads, tops[INT8 ? p : 0]);
    for (unsigned i = tid + kTops * kMoeThreads; i - r16 < n; i += kMoeThreads) look(i, __float_as_uint(a.g_max[i]));
  }
  auto place_group = [&]() {
    place_units();
    lds_barrier();
    place_cells();
#pragma unroll
    for (int p = 0; p < kScales; ++p) lds_put32(w0 + (tid + p * kMoeThreads) * 4, __float_as_uint(gs[p]));
    lds_barrier();
  };
  // (The first group by itself: its loads are ahead of the weights', and the waits
  // for them let the weights be on their way.)
  if (units != 0) place_group();
  while (g.u0 < units) {
    const MoeGroup cur = g;
    next_group();
    if (g.u0 < units) {   // the next group's, on their way while this one's units are multiplied
      load_cells(g.first, g.used);
      load_scales();
    }
    const MoeGroup ahead = g;
    g = cur;
    MoeUnit<TB, NB> now, next;
    if (mine < g.u1) load_unit(mine, now);
    for (; mine < g.u1; mine += kMoeWaves) {
      if (mine + kMoeWaves < g.u1) load_unit(mine + kMoeWaves, next);
      __builtin_amdgcn_s_waitcnt(0x0F70 | ((kSlots - 1) * NH));
      v8i w[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n)
        w[n] = 2 * n + 1 == NH ? lds_get2(h0 + read + n * 2048, h1 + read + n * 2048)
                               : lds_get2(f0 + read + n * 2048, f1 + read + n * 2048);
      read = read + kSlot == kSlots * kSlot ? 0 : read + kSlot;
      fetch();
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < TB; ++m) {
          if constexpr (INT8) {
            const v4i p = moe_mfma_int8(w[n], now.tok[m], v4i{0, 0, 0, 0});
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[m][n][r] = now.has[m] ? __builtin_fmaf((float)p[r], now.s[m] * now.sc[n][r], acc[m][n][r]) : acc[m][n][r];
          } else {
            const v4f p = moe_mfma_fp8(w[n], now.tok[m]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[m][n][r] = now.has[m] ? __builtin_fmaf(p[r], now.s[m] * now.sc[n][0], acc[m][n][r]) : acc[m][n][r];
          }
        }
      now = next;
    }
    g = ahead;
    if (g.u0 < units) {
      lds_barrier();   // the cells have been read
      place_group();
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // no direct load into LDS is left in flight
  __syncthreads();

  // ---- the wavefronts' sums, and the terms that are no expert's ----
  const unsigned sums = lds_at(ring_mem);
#pragma unroll
  for (int m = 0; m < TB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) lds_put(sums + ((wave * TB + m) * NB + n) * 1024 + lane * 16, acc[m][n]);
  __syncthreads();
  const float* part = reinterpret_cast<const float*>(ring_mem);
  for (int i = tid; i < 16 * NB * a.T; i += kMoeThreads) {
    const int token = i / (16 * NB), cc = i - token * 16 * NB, col = c0 + cc;
    if (cc >= cols) continue;
    const int m = token >> 4, n = cc >> 4;
    const int at = ((cc & 15) >> 2) * 64 + (token & 15) * 4 + (cc & 3);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kMoeWaves; ++w) v += part[((w * TB + m) * NB + n) * 256 + at];
    const int64_t o = (int64_t)token * H + col;
    // (what no route looks at may be infinite or NaN)
    const uint32_t has = tab.has[token];
    if (a.ori != nullptr && (has & 1)) v = __builtin_fmaf(tab.copy[token], __uint_as_float((uint32_t)a.ori[o] << 16), v);
    if (a.shared != nullptr && (has & 2)) v = __builtin_fmaf(tab.present[token], __uint_as_float((uint32_t)a.shared[o] << 16), v);
    a.out[o] = (uint16_t)bf16_rne(v);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Workspace: [status block][table][ids][scales][codes of x][their scales][g][g_max].
struct MoePlan {
  size_t off_table, off_ids, off_scales, off_q, off_q_scale, off_g, off_max, bytes;
};

MoePlan make_moe_plan(const mdc_shape* sh, int inter_n) {
  const size_t T = (size_t)sh->bs, R = T * sh->topk, H = (size_t)sh->hidden, N = (size_t)inter_n;
  MoePlan p;
  p.off_table = MDC_STATUS_BYTES;
  p.off_ids = p.off_table + round_up(sizeof(MoeTable), 256);
  p.off_scales = p.off_ids + round_up(R * 4, 256);
  p.off_q = p.off_scales + round_up(R * 4, 256);
  p.off_q_scale = p.off_q + round_up(T, 16) * H;
  p.off_g = p.off_q_scale + H / kFp8Block * kMoeTokens * 4;
  p.off_max = p.off_g + round_up(R * (N / 2) * 4, 256);
  p.bytes = p.off_max + round_up(R * (N / 16) * 4, 256);
  return p;
}

mdc_status check_moe(const mdc_shape* sh, int inter_n) {
  const mdc_status st = check_shape(sh);
  if (st != MDC_OK) return st;
  if (inter_n <= 0) return MDC_ERR_INVALID;
  if (inter_n % 256 != 0 || sh->hidden % kFp8Block != 0) return MDC_ERR_UNSUPPORTED;
  if (sh->bs > MDC_MAX_MOE_TOKENS || sh->hidden > kMoeWaves * kUpRun * kFp8Block) return MDC_ERR_UNSUPPORTED;
  if ((int64_t)inter_n * sh->hidden > INT32_MAX) return MDC_ERR_UNSUPPORTED;
  return MDC_OK;
}

template <typename T, int VPL>
void launch_prep(const Moe& a, GateArgs g, bool gated, bool int8, hipStream_t s) {
  g.vec = g.E % VPL == 0 && g.E * sizeof(T) % 16 == 0 && aligned16(g.logits) && aligned16(g.bias);
  const size_t lds = gated && g.groups > 1 && !gate_whole_lanes(g.E / g.groups, VPL) ? lds_slots(64, VPL) * sizeof(int64_t) : 0;
  hipLaunchKernelGGL((k_moe_prep<T, VPL>), dim3(a.T, gated ? 2 : 1), dim3(kPrepThreads), lds, s, a, g, int8 ? 1 : 0);
}

template <typename T>
void launch_prep_typed(const Moe& a, const GateArgs& g, bool int8, hipStream_t s) {
  if (g.E <= 64) launch_prep<T, 1>(a, g, true, int8, s);
  else if (g.E <= 128) launch_prep<T, 2>(a, g, true, int8, s);
  else if (g.E <= 256) launch_prep<T, 4>(a, g, true, int8, s);
  else if (g.E <= 512) launch_prep<T, 8>(a, g, true, int8, s);
  else if (g.E <= 1024) launch_prep<T, 16>(a, g, true, int8, s);
  else launch_prep<T, 32>(a, g, true, int8, s);
}

template <bool INT8, int TB>
void launch_moe(const Moe& a, unsigned cus, hipStream_t s) {
  hipLaunchKernelGGL((k_moe_up<INT8, TB>), dim3(cus), dim3(kMoeThreads), 0, s, a);
  const dim3 grid((unsigned)((a.H + a.cw - 1) / a.cw));
  const dim3 block(kMoeThreads);
  if (a.cw <= 8) hipLaunchKernelGGL((k_moe_down<INT8, TB, 1>), grid, block, 0, s, a);
  else if (a.cw <= 16) hipLaunchKernelGGL((k_moe_down<INT8, TB, 2>), grid, block, 0, s, a);
  else if (a.cw <= 24) hipLaunchKernelGGL((k_moe_down<INT8, TB, 3>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_moe_down<INT8, TB, 4>), grid, block, 0, s, a);
}

template <bool INT8>
mdc_status moe_impl(const mdc_shape* shape, const mdc_gate_params* params, int32_t inter_n, const void* x,
                    const void* logits, const float* bias, int32_t* expert_ids, float* expert_scales,
                    const uint8_t* x_active_mask, const void* w1, const float* w1_scale, const void* w2,
                    const float* w2_scale, const void* shared_expert_x, const void* ori_x, void* x_out, void* workspace,
                    size_t workspace_bytes, void* stream) {
  const mdc_status st = check_moe(shape, inter_n);
  if (st != MDC_OK) return st;
  const int64_t E = (int64_t)shape->num_experts + shape->zero_experts + shape->copy_experts;
  if (params != nullptr) {
    const mdc_status gate = check_gate(*params, E, shape->topk);
    if (gate != MDC_OK) return gate;
  }
  if (shape->bs == 0) return MDC_OK;   // (tensors of no tokens may be NULL, logits among them)
  if ((params != nullptr) != (logits != nullptr)) return MDC_ERR_NULLPTR;
  if ((expert_ids != nullptr) != (expert_scales != nullptr)) return MDC_ERR_NULLPTR;
  const MoePlan p = make_moe_plan(shape, inter_n);
  if (x == nullptr || w1 == nullptr || w1_scale == nullptr || w2 == nullptr || w2_scale == nullptr || x_out == nullptr ||
      workspace == nullptr || (params == nullptr && expert_ids == nullptr) ||
      (ori_x == nullptr && shape->copy_experts > 0 && shape->world == 1))
    return MDC_ERR_NULLPTR;
  if (!aligned16(x) || !aligned16(w1) || !aligned4(w1_scale) || !aligned16(w2) || !aligned4(w2_scale) ||
      !aligned16(shared_expert_x) || !aligned16(ori_x) || !aligned16(x_out) || !aligned16(workspace) ||
      !aligned4(expert_ids) || !aligned4(expert_scales) || !aligned4(bias) ||
      (params != nullptr && reinterpret_cast<uintptr_t>(logits) % (params->dtype == MDC_DTYPE_FP32 ? 4 : 2) != 0))
    return MDC_ERR_INVALID;
  if (workspace_bytes < p.bytes) return MDC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  if (expert_ids == nullptr) {
    expert_ids = reinterpret_cast<int32_t*>(ws + p.off_ids);
    expert_scales = reinterpret_cast<float*>(ws + p.off_scales);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const unsigned cus = device_cus();
  const int L = shape->num_experts / shape->world;
  const int cw = min(32, max(4, (int)round_up((shape->hidden + cus - 1) / cus, 4)));
  const Moe a{x, reinterpret_cast<uint8_t*>(ws + p.off_q), reinterpret_cast<float*>(ws + p.off_q_scale),
              reinterpret_cast<MoeTable*>(ws + p.off_table), expert_ids, expert_scales, x_active_mask, static_cast<const uint8_t*>(w1), w1_scale,
              static_cast<const uint8_t*>(w2), w2_scale, static_cast<const uint16_t*>(shared_expert_x),
              static_cast<const uint16_t*>(ori_x), static_cast<uint16_t*>(x_out), reinterpret_cast<float*>(ws + p.off_g),
              reinterpret_cast<float*>(ws + p.off_max), reinterpret_cast<mdc_device_status*>(ws), shape->bs, shape->topk,
              shape->hidden, inter_n, L, shape->rank * L, shape->num_experts,
              shape->num_experts + shape->zero_experts, shape->num_experts + shape->zero_experts + shape->copy_experts,
              shape->mask_per_route, cw};
  if (params != nullptr) {
    const GateArgs g{logits, bias, expert_ids, expert_scales, a.T, (int)E, a.K, params->groups, params->topk_groups,
                     params->group_top, params->score == MDC_GATE_SIGMOID, params->renormalise, params->scale, 0};
    if (params->dtype == MDC_DTYPE_BF16) launch_prep_typed<uint16_t>(a, g, INT8, s);
    else if (params->dtype == MDC_DTYPE_FP16) launch_prep_typed<_Float16>(a, g, INT8, s);
    else launch_prep_typed<float>(a, g, INT8, s);
  } else {
    launch_prep<float, 1>(a, GateArgs{}, false, INT8, s);
  }
  if (a.T <= 16) launch_moe<INT8, 1>(a, cus, s);
  else launch_moe<INT8, 2>(a, cus, s);
  return launched();
}

mdc_status moe_workspace(const mdc_shape* shape, int32_t inter_n, size_t* bytes) {
  if (bytes == nullptr) return MDC_ERR_NULLPTR;
  const mdc_status st = check_moe(shape, inter_n);
  if (st != MDC_OK) return st;
  *bytes = make_moe_plan(shape, inter_n).bytes;
  return MDC_OK;
}

}  // namespace

extern "C" {

mdc_status mdc_moe_workspace(const mdc_shape* shape, int32_t inter_n, size_t* bytes) {
  return moe_workspace(shape, inter_n, bytes);
}

mdc_status mdc_moe_fp8_workspace(const mdc_shape* shape, int32_t inter_n, size_t* bytes) {
  return moe_workspace(shape, inter_n, bytes);
}

mdc_status mdc_moe(const mdc_shape* shape, const mdc_gate_params* params, int32_t inter_n, const void* x,
                   const void* logits, const float* bias, int32_t* expert_ids, float* expert_scales,
                   const uint8_t* x_active_mask, const int8_t* w1, const float* w1_scale, const int8_t* w2,
                   const float* w2_scale, const void* shared_expert_x, const void* ori_x, void* x_out, void* workspace,
                   size_t workspace_bytes, void* stream) {
  return moe_impl<true>(shape, params, inter_n, x, logits, bias, expert_ids, expert_scales, x_active_mask, w1, w1_scale, w2,
                        w2_scale, shared_expert_x, ori_x, x_out, workspace, workspace_bytes, stream);
}

mdc_status mdc_moe_fp8(const mdc_shape* shape, const mdc_gate_params* params, int32_t inter_n, const void* x,
                       const void* logits, const float* bias, int32_t* expert_ids, float* expert_scales,
                       const uint8_t* x_active_mask, const void* w1, const float* w1_scale, const void* w2,
                       const float* w2_scale, const void* shared_expert_x, const void* ori_x, void* x_out, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return moe_impl<false>(shape, params, inter_n, x, logits, bias, expert_ids, expert_scales, x_active_mask, w1, w1_scale,
                         w2, w2_scale, shared_expert_x, ori_x, x_out, workspace, workspace_bytes, stream);
}

}  // extern "C"
