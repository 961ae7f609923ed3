// 4-bit expert weights with group scales: the quantizer, its inverse, and the expert
// products that read the codes directly.
//
// Format (w4.cuh): scale = max|v| / 7 over a group, rounded to 5 significant bits (1
// where that is below 2^-126), code = v / scale to the nearest whole number, ties to
// even, held as code + 8. |v| / scale is at most 7 (1 + 2^-5) < 7.5, so no code leaves
// [-7, 7]; and a code times a 5-bit scale has at most 8 significant bits, i.e. it IS a
// bf16 number: the value that a tensor core multiplies is the value the format stands
// for, whichever kernel reads it.
#include <algorithm>
#include <cstring>

#include "tc.cuh"
#include "w4.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------------ quantizer
// Both directions are bound by HBM when few instructions are spent an element: two bytes
// of weights and half a byte of codes each way.
constexpr int QW_WARPS = 8;    // warps a block
constexpr int QW_ROWS = 32;    // rows a turn of a block, 4 a warp
constexpr int QW_TURNS = 4;    // turns a block, at most
constexpr int QW_COLS = 256;   // columns a block: 8 a lane

__device__ __forceinline__ float scale_5bits(float amax) {
  uint32_t u = __float_as_uint(__fdiv_rn(amax, 7.f));
  u = (u + 0x3FFFFu + ((u >> 19) & 1u)) & 0xFFF80000u;  // nearest, ties to even, at mantissa bit 19
  return u >= 0x00800000u ? __uint_as_float(u) : 1.f;
}

// The bits of 1.5 2^23 + 8 + (v / scale to the nearest whole number, ties to even), with
// r = 1 / scale rounded: two instructions in place of a division. v has 8 significant bits
// and the scale 5, so v / scale is either exactly half-way between two whole numbers or at
// least 1 / 1280 from it. v r is off by at most 2^-21, so rounding it to multiples of
// 2^-12 first (the addition of 1.5 2^11) gives the half-way number exactly or stays on its
// side; the second addition rounds to whole numbers as the division would have.
__device__ __forceinline__ uint32_t code_bits(float v, float r) {
  constexpr float to_12 = 0x1.8p11f, to_0 = 0x1.8p23f + 8.f - to_12;
  return __float_as_uint(__fadd_rn(__fmaf_rn(v, r, to_12), to_0));
}

__device__ __forceinline__ uint32_t abs_max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b & 0x7FFF7FFFu));
  return d;
}

// A block takes QW_COLS columns of QW_TURNS x QW_ROWS rows: a lane 8 columns of 4 rows a
// turn, the next turn's loads in flight meanwhile. The group's maximum comes from the
// G / 8 lanes that share it (two rows in one register); the scales meet in shared memory
// so that each group's scales leave as one run of the group-major layout.
template <int G>
__global__ void __launch_bounds__(QW_WARPS * 32)
    quantize_w4_kernel(int rows, int cols, int turns, const uint4* __restrict__ src, uint32_t* __restrict__ codes,
                       __nv_bfloat16* __restrict__ scales) {
  constexpr int GPB = QW_COLS / G, ROWS = QW_ROWS * QW_TURNS;
  __shared__ __nv_bfloat16 sc_s[GPB][ROWS];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long mat = blockIdx.z;
  const int ng = (cols + G - 1) / G;
  const int c8 = blockIdx.x * (QW_COLS / 8) + lane, n8 = cols >> 3;
  const int row_b = blockIdx.y * turns * QW_ROWS;
  const bool cok = c8 < n8;
  auto fetch = [&](uint4 (&v)[4], const int turn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = row_b + turn * QW_ROWS + warp * 4 + i;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (cok && row < rows) v[i] = __ldcs(src + (mat * rows + row) * n8 + c8);
    }
  };
  uint4 v[4], nx[4];
  fetch(v, 0);
#pragma unroll 1
  for (int turn = 0; turn < turns; ++turn) {
    const int row0 = row_b + turn * QW_ROWS + warp * 4;
    if (row_b + turn * QW_ROWS >= rows) break;
    if (turn + 1 < turns) fetch(nx, turn + 1);
    uint32_t m[2];  // the maxima of rows 0, 1 and 2, 3
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t a = 0u, b = 0u;
      a = abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(a, v[2 * i].x), v[2 * i].y), v[2 * i].z),
                         v[2 * i].w);
      b = abs_max_bf16x2(
          abs_max_bf16x2(abs_max_bf16x2(abs_max_bf16x2(b, v[2 * i + 1].x), v[2 * i + 1].y), v[2 * i + 1].z),
          v[2 * i + 1].w);
      m[i] = abs_max_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
      for (int off = G / 16; off > 0; off >>= 1) m[i] = abs_max_bf16x2(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
    }
    // lane i of a group's lanes works out row i % 4's scale for all of them
    const uint32_t mine = lane & 2 ? m[1] : m[0];
    const float sc = scale_5bits(__uint_as_float(lane & 1 ? mine & 0xFFFF0000u : mine << 16)), rc = __frcp_rn(sc);
    if (lane % (G / 8) < 4) sc_s[lane / (G / 8)][turn * QW_ROWS + warp * 4 + (lane & 3)] = __float2bfloat16_rn(sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float r = __shfl_sync(0xffffffffu, rc, (lane & ~3) + i);
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      // each term is 0x4B400000 + code + 8: the sum of the shifted terms less the shifted constants
      uint32_t word = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        word += (code_bits(__uint_as_float(w[j] << 16), r) << (4 * j)) +
                (code_bits(__uint_as_float(w[j] & 0xFFFF0000u), r) << (16 + 4 * j));
      if (cok && row0 + i < rows) codes[(mat * rows + row0 + i) * n8 + c8] = word;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = nx[i];
  }
  __syncthreads();
  const int n = turns * QW_ROWS;  // rows of this block: a power of two
  for (int i = threadIdx.x; i < GPB * n; i += QW_WARPS * 32) {
    const int gl = i / n, r = i % n, g = blockIdx.x * GPB + gl, row = row_b + r;
    if (g < ng && row < rows) scales[(mat * ng + g) * rows + row] = sc_s[gl][r];
  }
}

// bf16 pair of the codes at bits 0..3 and 16..19 of w, minus 8: the bf16 number with
// exponent bits 0x4300 and the code in its last mantissa bits is 128 + code, and the
// difference to 136 is exact.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(0x000F000Fu), "r"(0x43004300u));  // (w & a) | b
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(r), "r"(0x43084308u));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The same times a scale s, in one rounding and one instruction less: bf16 with exponent
// bits 0x4180 and the code at mantissa bit 3 is 16 + code, and (16 + code) s - 24 s is
// rounded once. This needs 24 s to be a bf16 number: w4_scale_is_short says that s has at
// most 6 significant bits (the quantizer's have 5) and is not so large that 24 s overflows.
// (The lowest pair needs no shift the other way: two products on the FMA pipe for a shift
// on the ALU pipe, which the unpacking loads more.)
__device__ __forceinline__ uint32_t w4_pair_scaled(uint32_t w, int e, uint32_t ss, uint32_t ms) {
  if (e == 0) return mul_bf16x2(w4_pair(w), ss);
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
      : "=r"(r)
      : "r"(w >> (4 * e - 3)), "r"(0x00780078u), "r"(0x41804180u));  // (w & a) | b
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(r), "r"(ss), "r"(ms));
  return d;
}
__device__ __forceinline__ bool w4_scale_is_short(uint32_t s) { return (s & 3u) == 0u && (s & 0x7FFFu) < 0x7C00u; }

// The inverse: bf16(code * scale) (exact for the quantizer's scales). A lane turns one
// word (8 columns) of 4 neighbouring rows a turn into 16 bytes each, the next turn's words
// in flight meanwhile.
template <int G>
__global__ void __launch_bounds__(QW_WARPS * 32)
    dequantize_w4_kernel(int rows, int cols, int turns, const uint32_t* __restrict__ codes,
                         const uint16_t* __restrict__ scales, uint4* __restrict__ dst) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long mat = blockIdx.z;
  const int ng = (cols + G - 1) / G;
  const int c8 = blockIdx.x * (QW_COLS / 8) + lane, n8 = cols >> 3;
  const int row_b = blockIdx.y * turns * QW_ROWS + warp * 4;
  if (c8 >= n8) return;
  uint32_t w[4], nw[4];
  uint2 s4, ns4;
  auto fetch = [&](uint32_t (&d)[4], uint2& s, const int turn) {
    const int row0 = row_b + turn * QW_ROWS;
    if (turn >= turns || row0 >= rows) return;  // rows % 8 == 0: the 4 rows exist together
    s = *reinterpret_cast<const uint2*>(scales + (mat * ng + 8 * c8 / G) * rows + row0);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = __ldcs(codes + (mat * rows + row0 + i) * n8 + c8);
  };
  fetch(w, s4, 0);
#pragma unroll 1
  for (int turn = 0; turn < turns; ++turn) {
    const int row0 = row_b + turn * QW_ROWS;
    if (row0 >= rows) break;
    fetch(nw, ns4, turn + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = ((i & 2) ? s4.y : s4.x) >> (16 * (i & 1)) & 0xFFFFu, ss = h | (h << 16);
      uint4 o;
      o.x = mul_bf16x2(w4_pair(w[i]), ss);
      o.y = mul_bf16x2(w4_pair(w[i] >> 4), ss);
      o.z = mul_bf16x2(w4_pair(w[i] >> 8), ss);
      o.w = mul_bf16x2(w4_pair(w[i] >> 12), ss);
      __stcs(dst + (mat * rows + row0 + i) * n8 + c8, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = nw[i];
    s4 = ns4;
  }
}

// ------------------------------------------------------------------ expert products
// out rows = epi(rows of x . W_g^T), every group in one persistent launch, on the
// 5th-generation tensor cores.
//
// The weights are the matrix instruction's A operand (M = 128 rows a CTA), the segment's
// input rows its B operand (N = up to BN), so a few rows waste no M tile. The codes travel
// as they are, HBM -> shared memory (TMA); groups of four warps turn them into bf16 values
// (code - 8 is exact in bf16, times the scale is one rounding, none for the quantizer's
// scales) and put them straight into TENSOR MEMORY, from where the matrix instruction
// takes its A operand. So the expanded weights never touch shared memory: per 128 columns
// of K it sees 9 KB of codes and scales and the input rows, where bf16 tiles of the same
// shape would bring 32 KB of weights more.
//
// Tile: 128 weight rows (PAIR, long segments: 256 over two CTAs, which then read half of
// the input rows each) x up to BN input rows x the whole K. SwiGLU tiles hold half as many
// features: of a CTA's 128 rows, lane quarter q (32 lanes of tensor memory) holds 16 gate
// rows, then the same features' 16 up rows, so one shuffle across 16 lanes brings a
// feature's two sums together and one accumulator serves both matrices.
//
// Schedule (device side, from the segment offsets): the tiles of all groups, tallest
// first. Whole tiles go round the walkers (CTAs or pairs) in alternating direction, so
// that those working at the same time share an expert's rows in L2; the last one to two
// rounds (everything, when there are fewer tiles than walkers, as in decode) are cut into
// equal runs of chunks of K, one a walker. A tile cut between walkers is joined through
// fp32 partial sums in the workspace: whichever warp finishes last adds them in the order
// of K, so the result does not depend on who that is, and no one waits.
//
// Warps: 0 and 2 TMA producers (codes and scales; input rows), 1 (and 3) matrix issuers
// (PAIR: in the leader CTA), 1 also owner of the tensor memory, then teams of four that take
// turns to expand chunks, then the epilogue's. The issuer's instruction stream is what bounded
// the first forms of this kernel (a ready barrier costs it 84 cycles, a product 20, a
// commit 46, and some hundred a turn of a long loop), so it commits once a chunk.
// Barriers of a stage of the ring: codes (local) -> expanders; input rows (PAIR: of both
// CTAs, at the leader) -> issuer; expanded (PAIR: at the leader) -> issuer; free: the
// issuer's commit. A slot in tensor memory is free once the chunk A_SLOTS before is done,
// which that chunk's stage barrier tells. Every wait is bounded in time as in tc_gemm.cu.
constexpr int WT_EXPAND_WARP = 4;
constexpr int WT_MAX_GROUPS = 1040;
constexpr unsigned long long WT_DRAIN_LIMIT_NS = 200ull * 1000 * 1000;

template <int BN>
struct WtShape {
  static constexpr bool PAIR = BN >= 64;
  static constexpr int PHASES = BN <= 64 ? 2 : 1;      // both products in one launch
  static constexpr int SMEM_BUDGET = (PHASES == 2 ? 180 : 196) * 1024;
  static constexpr int BK = BN > 64 ? 128 : 256;       // columns of K a stage
  static constexpr int TEAMS = BN > 128 || BN == 32 || BN == 64 ? 2 : 3;    // teams of four expanding warps
  static constexpr int EW = BN > 128 ? 8 : 4;              // epilogue warps
  static constexpr int EPI_WARP = WT_EXPAND_WARP + 4 * TEAMS;
  static constexpr int THREADS = 32 * (EPI_WARP + EW);
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;    // input rows a CTA
  static constexpr int HALF = B_ROWS / 2;               // staged rows where half of a CTA's suffice
  static constexpr int X_SUB = B_ROWS * 128;           // 64 columns of K: 128-byte rows
  static constexpr int X_BYTES = BK / 64 * X_SUB;
  static constexpr int CODE_BYTES = 128 * BK / 2;
  static constexpr int SCALE_BYTES = 128 * 2 * BK / 32;  // at most, groups of 32
  static constexpr int STAGE_BYTES = X_BYTES + CODE_BYTES + SCALE_BYTES;
  static constexpr int STAGES_RAW = SMEM_BUDGET / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 12 ? 12 : STAGES_RAW;
  // Issuers: short segments have two (in warps 1 and 3) that take alternate chunks, each
  // with a sum of its own, since one's instruction stream would set the pace.
  static constexpr int ISSUERS = PAIR ? 1 : 2;
  // Two sums in tensor memory, so that a tile's epilogue runs beside the next tile's
  // products; one for the tallest tiles, whose long K hides it (w4_deep).
  static constexpr int NUM_ACC = BN > 192 ? 1 : 2, ACC_COLS = ISSUERS * BN;
  // Expanded weights in tensor memory: a ring of slots of a chunk (two bf16 a column). A
  // slot is free once the chunk A_SLOTS before is done.
  static constexpr int A_COLS = BK / 2;
  static constexpr int A_SLOTS_RAW = (512 - NUM_ACC * ACC_COLS) / A_COLS;
  static constexpr int A_SLOTS = A_SLOTS_RAW > STAGES - TEAMS ? STAGES - TEAMS : A_SLOTS_RAW;
  static constexpr int DYN_SMEM = STAGES * STAGE_BYTES + 1024;
  static_assert(BN % 16 == 0 && BN >= 16 && BN <= 256 && HALF % 8 == 0, "tile");
  static_assert(STAGE_BYTES % 1024 == 0 && A_SLOTS >= 2, "ring");
  // A wait tells a barrier's phases apart by parity alone, so whoever waits for chunk n in
  // a stage must know that chunk n - STAGES, the stage's last, has passed there. What is
  // known: an issuer is done with its chunks in order, and a chunk was expanded when the
  // chunk A_SLOTS before it was done. So a team at chunk n knows from its turn before that
  // chunk m = n - TEAMS - A_SLOTS is done, with it m - A_SLOTS, and of one issuer all, of
  // two every second chunk before those: any but m - 1. An issuer at chunk n knows its own
  // earlier ones, and from its last that chunk n - ISSUERS - A_SLOTS is done.
  static_assert(STAGES >= TEAMS + A_SLOTS && (ISSUERS == 1 || STAGES != TEAMS + A_SLOTS + 1), "expanders' phases");
  static_assert(ISSUERS == 1 || (A_SLOTS == 3 && (STAGES % 2 == 0 || STAGES == 5)), "issuers' phases");
};

template <int PHASES>
struct WtMaps {
  CUtensorMap codes[2 * PHASES][2], scales[2 * PHASES][2];  // [phase, class][matrix]
  CUtensorMap x[2 * PHASES][2];  // [class][half]: 64 columns x B_ROWS (HALF) rows x BK / 64
  CUtensorMap xt[2 * PHASES];    // 64 columns x HALF rows, columns behind K as zero
};

// A piece of work: chunks [c0, c1) of K of one tile. cls: 2 phase + class.
struct alignas(16) WtItem {
  int cls, g, mt, rows, b_row, out_row, c0, c1;
  int wa, wb;  // walkers that share the tile
  int pad[2];
};

constexpr int WT_ITEMS = 96;  // pieces of a walker that are worked out before it starts

struct WtPhase {
  int tile_start[WT_MAX_GROUPS + 1];  // groups in walk order: first tile
  int cost[WT_MAX_GROUPS + 1];        // and cost of the cut tiles before
  int rounds, t0;   // rounds of whole tiles; first cut tile
  int cut, per;     // cost of the cut tiles, of a walker's share
  int t_first, n;   // this walker's first cut tile, all its pieces
};

template <int PHASES>
struct WtSched {
  WtPhase ph[PHASES];
  int gid[WT_MAX_GROUPS];
  int rows[WT_MAX_GROUPS], brow[WT_MAX_GROUPS];  // by group; first row in its segment order
  short height[WT_MAX_GROUPS];
  int hist[32];
  int none;  // no work: an error that was there before the launch, or bad offsets
  WtItem items[WT_ITEMS];
};

template <int BN>
__device__ __forceinline__ int wt_height(int rows) {
  const int nt = (rows + BN - 1) / BN;
  return nt > 0 ? min(BN, (((rows + nt - 1) / nt) + 15) & ~15) : 0;
}
// Cost of a chunk of a tile of `height` rows: the matrix instruction's time, at least
// that of expanding the codes (as long as 64 rows take).
__device__ __forceinline__ int wt_weight(int height) { return max(height >> 4, 4); }

template <int BN>
__device__ __forceinline__ int wt_chunks(const W4Class& c) {
  return (c.K + WtShape<BN>::BK - 1) / WtShape<BN>::BK;
}

// Largest position whose entry is at most v (entries ascend, the first is at most v).
__device__ __forceinline__ int wt_find(const int* e, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (e[mid] <= v) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Output features of a tile in a phase: of SwiGLU's first product half a tile's rows.
template <int BN, int EPI>
__device__ __forceinline__ int wt_cta_f(int phase) {
  return EPI == EPI_SWIGLU && phase == 0 ? 64 : 128;
}

// Piece i of a walker, over all phases; a cut tile may leave it an empty one.
template <int BN>
__device__ __forceinline__ WtItem wt_item(const W4Params& p, const WtSched<WtShape<BN>::PHASES>& s, int G, int walker,
                                          int walkers, int i) {
  WtItem it;
  int phase = 0;
  if (WtShape<BN>::PHASES == 2 && i >= s.ph[0].n) {
    phase = 1;
    i -= s.ph[0].n;
  }
  const WtPhase& f = s.ph[phase];
  const bool whole = i < f.rounds;
  const int tile = whole ? i * walkers + ((i & 1) ? walkers - 1 - walker : walker) : f.t_first + i - f.rounds;
  const int pos = wt_find(f.tile_start, G, tile);
  const int gi = s.gid[pos], G0 = p.cls[0].n_groups, cl = gi < G0 ? 0 : 1;
  it.cls = 2 * phase + cl;
  it.g = gi - (cl ? G0 : 0);
  const W4Class& c = p.cls[it.cls];
  const int rows = s.rows[gi], NT = (rows + BN - 1) / BN, h = s.height[gi];
  const int local = tile - f.tile_start[pos], nt = local % NT, nc = wt_chunks<BN>(c);
  it.mt = local / NT;
  it.rows = min(h, rows - nt * h);
  it.b_row = (c.seg_off ? s.brow[gi] : it.g * c.b_group_stride) + nt * h;
  it.out_row = (c.seg_off ? s.brow[gi] : it.g * c.out_group_stride) + nt * h;
  it.c0 = 0;
  it.c1 = nc;
  it.wa = it.wb = walker;
  if (!whole) {
    // chunk j of the tile costs w and starts at `at` + j w: it is walker (that / per)'s
    const int w = wt_weight(h), at = f.cost[pos] + (tile - max(f.tile_start[pos], f.t0)) * nc * w;
    const int lo = walker * f.per, hi = min(lo + f.per, f.cut);
    it.c0 = lo > at ? (lo - at + w - 1) / w : 0;
    it.c1 = min(nc, (hi - at + w - 1) / w);
    it.wa = at / f.per;
    it.wb = (at + (nc - 1) * w) / f.per;
  }
  return it;
}

// The schedule, by one warp: groups ordered by tile height, tallest first (a counting
// sort over the heights, stable in group order), tiles and costs added up in that order,
// and this walker's first pieces of work. First the order, then a warp for each phase.
//
// The CTAs of a launch share tiles, so all of them must lay out the same schedule. Each
// checks every offset for itself, and any bad one leaves it without work: were that left to
// the status word (`prior`, read before), only CTAs that read it after another's check
// would stop.
template <int BN>
__device__ __forceinline__ void wt_order(const W4Params& p, WtSched<WtShape<BN>::PHASES>& s, int G, int lane,
                                         int prior) {
  constexpr int NB = BN / 16 + 1;  // bucket = tile height / 16 (0: a group without rows)
  static_assert(NB <= 32, "a bucket a lane");
  const int G0 = p.cls[0].n_groups;
  bool bad = prior != 0;
  s.hist[lane] = 0;
  __syncwarp();
  for (int g0 = 0; g0 < G; g0 += 32) {
    const int gi = g0 + lane;
    int key = -1;
    if (gi < G) {
      const int cl = gi < G0 ? 0 : 1, g = gi - (cl ? G0 : 0);
      const W4Class& c = p.cls[cl];
      int rows, brow;
      if (c.seg_off) {
        const int a = c.seg_off[g], b = c.seg_off[g + 1];
        rows = b - a;
        brow = a;
        if (a < 0 || b < a || b > c.max_row) {
          set_status(p.status, MOE_ERR_DEVICE_INDEX);
          bad = true;
          rows = brow = 0;
        }
      } else {
        rows = c.const_rows;
        brow = 0;
      }
      const int h = wt_height<BN>(rows);
      key = h >> 4;
      s.rows[gi] = rows;
      s.brow[gi] = brow;
      s.height[gi] = (short)h;
    }
    // rank among the groups of this height so far
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int before = 0;
    if (key >= 0) before = s.hist[key];
    __syncwarp();
    if (key >= 0 && rank == 0) s.hist[key] = before + __popc(same);
    if (gi < G) s.ph[0].cost[gi] = before + rank;
    __syncwarp();
  }
  {  // first position of each height, tallest first
    const int n = lane < NB ? s.hist[NB - 1 - lane] : 0;
    int inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += v;
    }
    __syncwarp();
    if (lane < NB) s.hist[NB - 1 - lane] = inc - n;
    __syncwarp();
  }
  for (int gi = lane; gi < G; gi += 32) s.gid[s.hist[s.height[gi] >> 4] + s.ph[0].cost[gi]] = gi;
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) s.none = bad;
  __syncwarp();
}

template <int BN, int EPI>
__device__ __forceinline__ void wt_phase(const W4Params& p, WtSched<WtShape<BN>::PHASES>& s, int G, int walker,
                                         int walkers, int lane, int phase) {
  using S = WtShape<BN>;
  WtPhase& f = s.ph[phase];
  const int G0 = p.cls[0].n_groups;
  const int log2_f = (EPI == EPI_SWIGLU && phase == 0 ? 6 : 7) + (S::PAIR ? 1 : 0);
  const int tiles0 = (p.cls[2 * phase].R + (1 << log2_f) - 1) >> log2_f;
  const int tiles1 = (p.cls[2 * phase + 1].R + (1 << log2_f) - 1) >> log2_f;
  const int nc0 = wt_chunks<BN>(p.cls[2 * phase]), nc1 = wt_chunks<BN>(p.cls[2 * phase + 1]);
  const int per = (G + 31) / 32, lo = min(G, lane * per), hi = min(G, lo + per);
  int sum = 0;
  for (int pos = lo; pos < hi; ++pos) {
    const int gi = s.gid[pos], n = (gi < G0 ? tiles0 : tiles1) * ((s.rows[gi] + BN - 1) / BN);
    f.tile_start[pos] = sum;  // (this lane's part)
    sum += n;
  }
  int inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  for (int pos = lo; pos < hi; ++pos) f.tile_start[pos] += inc - sum;
  int total = __shfl_sync(0xffffffffu, inc, 31);
  if (lane == 0) f.tile_start[G] = total;
  __syncwarp();
  if (s.none) total = 0;
  // whole rounds, and the tiles that are cut
  int rounds = 0;
  if (total >= walkers) {
    rounds = total / walkers;
    if (rounds * walkers != total) --rounds;
  }
  const int t0 = rounds * walkers;
  sum = 0;
  for (int pos = lo; pos < hi; ++pos) {
    const int gi = s.gid[pos], n = f.tile_start[pos + 1] - max(f.tile_start[pos], t0);
    f.cost[pos] = sum;
    if (n > 0 && total) sum += n * (gi < G0 ? nc0 : nc1) * wt_weight(s.height[gi]);
  }
  inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  for (int pos = lo; pos < hi; ++pos) f.cost[pos] += inc - sum;
  const int cut = __shfl_sync(0xffffffffu, inc, 31);
  __syncwarp();
  // (at least 512 columns of the heaviest tile, so that every walker between a tile's
  // first and last one has a part of it)
  const int share = max((cut + walkers - 1) / walkers, 512 / S::BK * max(BN / 16, 4));
  const int from = walker * share, to = min(from + share, cut);
  int tile = 0;
  if (lane < 2 && from < to) {  // the tiles that hold the first and the last of its cost
    const int x = lane == 0 ? from : to - 1;
    const int pos = wt_find(f.cost, G, x), gi = s.gid[pos];
    tile = max(f.tile_start[pos], t0) + (x - f.cost[pos]) / ((gi < G0 ? nc0 : nc1) * wt_weight(s.height[gi]));
  }
  const int last = __shfl_sync(0xffffffffu, tile, 1);
  if (lane == 0) {
    f.rounds = rounds;
    f.t0 = t0;
    f.cut = cut;
    f.per = share;
    f.t_first = tile;
    f.n = rounds + (from < to ? last - tile + 1 : 0);
  }
  __syncwarp();
  if (S::PHASES == 1)
    for (int i = lane; i < min(f.n, WT_ITEMS); i += 32) s.items[i] = wt_item<BN>(p, s, G, walker, walkers, i);
}

// The list of a walker's pieces of work, walked alike by every role.
template <int BN>
struct WtWalk {
  const W4Params& p;
  const WtSched<WtShape<BN>::PHASES>& s;
  int G, walker, walkers, i, n;

  __device__ __forceinline__ WtWalk(const W4Params& p_, const WtSched<WtShape<BN>::PHASES>& s_, int G_, int w, int ws)
      : p(p_), s(s_), G(G_), walker(w), walkers(ws), i(0), n(-1) {}

  __device__ __forceinline__ int all() const {
    return s.ph[0].n + (WtShape<BN>::PHASES == 2 ? s.ph[WtShape<BN>::PHASES - 1].n : 0);
  }
  __device__ __forceinline__ bool next(WtItem& it) {
    if (n < 0) n = all();
    while (i < n) {
      it = i < WT_ITEMS ? s.items[i] : wt_item<BN>(p, s, G, walker, walkers, i);
      ++i;
      if (it.c0 < it.c1) return true;
    }
    return false;
  }
};

// Waits (bounded) until the grid's count has reached `target`, then orders what the counted
// warps stored before the copies that this warp issues next.
__device__ __forceinline__ bool w4_grid_wait(unsigned long long* count, unsigned long long target,
                                             unsigned long long limit_ns, const volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  bool ok = true;
  while (true) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(count) : "memory");
    if (__all_sync(0xffffffffu, v >= target)) break;
    if (__any_sync(0xffffffffu, *abort_flag != 0 || globaltimer_ns() - t0 > limit_ns)) {
      ok = false;
      break;
    }
  }
  __threadfence();
  asm volatile("fence.proxy.async.global;" ::: "memory");
  __syncwarp();
  return ok;
}

// D (+)= A . B^T, A in tensor memory (PAIR: over both CTAs).
template <bool PAIR>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrive on the barrier (PAIR: at this offset in both CTAs) once every product so far completed.
template <bool PAIR>
__device__ __forceinline__ void umma_commit_all(uint64_t* bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    umma_commit(bar);
}
__device__ __forceinline__ void tmem_st_x32(uint32_t t, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

// Barrier of the two warps that lay out the schedule of two products (named barrier 1).
__device__ __forceinline__ void schedule_bar() { asm volatile("barrier.sync 1, 64;" ::: "memory"); }

// Bytes that a barrier expects and no copy will bring, counted as if one had.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}
// A word of a CTA of the pair, read from or written to it (a shared::cluster address).
__device__ __forceinline__ uint32_t ld_cluster(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// What a role does whose wait ran out, or that another role's tells to stop (PAIR: both
// CTAs' settle words are set). Not inlined, like wt_settle: a launch of microseconds starts
// with a cold instruction cache.
template <bool PAIR>
__device__ __noinline__ void wt_give_up(int* status, volatile int* abort_flag, uint32_t settle) {
  set_status(status, MOE_ERR_TIMEOUT);
  *abort_flag = 1;
  if (PAIR)
    for (uint32_t r = 0; r < 2; ++r) st_cluster(mapa_shared(settle, r), 1u);
}

// The leader CTA of a pair in which a role gave up waits for both CTAs' input rows. Rows
// that one CTA fetched (chunks used[0], the stages whose last copy was the short one
// used[1]) and the other did not: stage by stage the barrier gets the expectation, or the
// bytes, that it lacks. A stage is fetched again only after a product has read it, so it
// lacks at most its last fill.
template <int STAGES>
__device__ __noinline__ void wt_settle(uint64_t* x_full, const int* used, uint32_t bytes_half, uint32_t bytes_full) {
  const uint32_t peer_used = mapa_shared(smem_u32(used), 1u);
  const int own = used[0], peer = (int)ld_cluster(peer_used), last = max(own, peer);
  const uint32_t halves = own > peer ? (uint32_t)used[1] : ld_cluster(peer_used + 4);
  for (int n = min(own, peer); n < last; ++n) {
    const int i = n % STAGES;
    const uint32_t bytes = (halves >> i & 1u) ? bytes_half : bytes_full;
    if (own > peer)
      mbar_complete_tx(&x_full[i], bytes);
    else
      mbar_arrive_expect_tx(&x_full[i], bytes);
  }
  for (int i = 0; i < STAGES && i < last; ++i) {
    const volatile int never = 0;
    mbar_wait(&x_full[i], (uint32_t)((last - 1 - i) / STAGES) & 1u, WT_DRAIN_LIMIT_NS, &never);
  }
}

// Tile copy over three dimensions; PAIR: counted on a barrier of the leader CTA.
template <bool PAIR>
__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint32_t bar, void* dst, int x, int y, int z) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

template <int BN, int EPI>
__global__ void __launch_bounds__(WtShape<BN>::THREADS, 1)
    w4_gemm_kernel(const __grid_constant__ WtMaps<WtShape<BN>::PHASES> maps, const __grid_constant__ W4Params p) {
  using S = WtShape<BN>;
  constexpr bool PAIR = S::PAIR, TWO = S::PHASES == 2;
  constexpr int CTAS = PAIR ? 2 : 1;
  constexpr int STAGES = S::STAGES, A_SLOTS = S::A_SLOTS, BK = S::BK, EW = S::EW;
  __shared__ WtSched<S::PHASES> sched;
  __shared__ __align__(8) uint64_t code_full[STAGES], x_full[STAGES], a_full[STAGES], stage_free[STAGES],
      acc_full[2], acc_free[2], drain_bar;
  __shared__ __align__(16) __nv_bfloat16 stg[EPI == EPI_DOWN ? 1 : EW][16][32];  // epilogue warp: 16 output rows
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  // PAIR: chunks whose input rows this CTA fetched and the stages whose last such copy was
  // the short one; whether a role of either CTA gave up
  __shared__ int x_used_s[2], settle_s;
  __shared__ unsigned long long launch_s;  // TWO: the launch's number on this workspace
  extern __shared__ uint8_t dyn_smem[];

  // (the shuffle tells the compiler that the role is the whole warp's: loop state and
  // descriptors then live in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int walker = PAIR ? (int)cluster_id_x() : (int)blockIdx.x;
  const int walkers = PAIR ? (int)nclusters_x() : (int)gridDim.x;
  const uint32_t smem_base = (smem_u32(dyn_smem) + 1023u) & ~1023u;
  uint8_t* smem_gen = dyn_smem + (smem_base - smem_u32(dyn_smem));
  const int G0 = p.cls[0].n_groups, G = G0 + (p.n_classes > 1 ? p.cls[1].n_groups : 0);
  volatile int* abort_flag = &abort_s;
  const auto give_up = [&]() { wt_give_up<PAIR>(p.status, abort_flag, smem_u32(&settle_s)); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&x_full[i], 1);
      mbar_init(&a_full[i], 4 * CTAS + (p.stall == 1));  // a team of each CTA
      mbar_init(&stage_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], S::ISSUERS);
      mbar_init(&acc_free[i], EW * CTAS);  // the epilogue warps of each CTA
    }
    mbar_init(&drain_bar, S::ISSUERS);
    abort_s = 0;
    settle_s = 0;
    fence_mbar_init();
  }
  if (warp == 2 && lane < (int)(sizeof(maps) / sizeof(CUtensorMap)))
    tma_prefetch_desc(reinterpret_cast<const CUtensorMap*>(&maps) + lane);
  if (warp == 1) {
    tmem_alloc_g<PAIR>(&tmem_base_s, 512);
    tmem_relinquish_g<PAIR>();
  }
  __syncwarp();
  pdl_launch_dependents();
  tc_fence_before();
  if (PAIR)
    cluster_sync_all();  // the peer's barriers are initialised before either CTA signals them
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  // Barriers and tensor memory are ready. Warp 0 (and 2) waits for the kernels before this
  // one and lays out the schedule, warp 3 sees to the counters; the expanders run their loop body
  // once on whatever the shared memory holds, which fetches its instructions meanwhile.
  if (warp == 0 || (TWO && warp == 2)) {
    pdl_wait();
    // an earlier kernel of the call that flagged a device error leaves tables that are not used
    if (warp == 0) wt_order<BN>(p, sched, G, lane, p.status ? *reinterpret_cast<volatile int*>(p.status) : 0);
    __syncwarp();
    if (TWO) schedule_bar();
    wt_phase<BN, EPI>(p, sched, G, walker, walkers, lane, warp >> 1);
    if (TWO) {
      schedule_bar();
      const int n0 = sched.ph[0].n, n = n0 + sched.ph[S::PHASES - 1].n;
      for (int i = (warp ? n0 : 0) + lane; i < min(warp ? n : n0, WT_ITEMS); i += 32)
        sched.items[i] = wt_item<BN>(p, sched, G, walker, walkers, i);
    }
    __syncwarp();
  } else if (warp == 3) {
    // TWO: the second product's input rows are the first one's output, so they wait for a
    // grid-wide count of the epilogue warps that have left the first product (all CTAs are
    // resident: a cooperative launch). The count only grows, by W4_COUNT a launch whatever
    // happens in it (its first warp adds what the others' ones leave of that), so launches
    // are numbered by it. (The weights do not wait: the ring holds the second product's
    // first chunks before the last CTA leaves the first.)
    // The counters of cut tiles: this launch zeroes the set that the next one uses,
    // whatever a launch that was cut short has left there.
    pdl_wait();
    if (TWO) {
      unsigned long long v;
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p.grid_count) : "memory");
      const unsigned long long number = v / W4_COUNT;
      if (lane == 0) launch_s = number;
      if (blockIdx.x == 0)
        for (int i = lane; i < 2 * W4_COUNTERS2; i += 32)
          p.counters[(number & 1 ? 0 : 2 * W4_COUNTERS2) + i] = 0u;
    } else if (blockIdx.x == 0) {
      for (int i = lane; i < W4_COUNTERS; i += 32) p.counters_next[i] = 0u;
    }
  }
  if (warp < WT_EXPAND_WARP || warp >= S::EPI_WARP) __syncthreads();  // the schedule is there
  const unsigned long long lim = p.wait_limit_ns;
  WtWalk<BN> walk(p, sched, G, walker, walkers);
  WtItem it;
  bool ok = true;

  if (warp == 0 || warp == 2) {
    // ---------------------------------------------------------------- producers
    // Warp 0 fetches codes and scales, warp 2 the input rows (one warp's issue slots
    // would bound the short tiles). As in the issuer, the whole warp walks and waits and
    // one lane issues.
    const bool codes = warp == 0;
    if (!codes && p.stall == 2 + rank) walk.n = min(walk.all(), 1);
    bool second = false;
    int st = 0, used = 0;
    uint32_t ph = 0, halves = 0;
    const int gpc = BK / p.group;
    while (ok && walk.next(it)) {
      const W4Class& c = p.cls[it.cls];
      const int cta_f = wt_cta_f<BN, EPI>(it.cls >> 1);
      const bool mats2 = cta_f == 64;
      const int K = c.K, f0 = (it.mt * CTAS + (int)rank) * cta_f;
      const bool live = f0 < c.R;  // a CTA whose rows lie behind the matrix loads no weights
      const int y = it.g * c.R + f0, ys = it.g * ((K + p.group - 1) / p.group);
      const int cta_rows = ((it.rows + 15) & ~15) / CTAS;
      const bool half = cta_rows <= S::HALF;
      if (TWO && !codes && it.cls >= 2 && !second) {
        second = true;
        if (!w4_grid_wait(p.grid_count, (launch_s + 1) * W4_COUNT, lim, abort_flag)) {
          ok = false;
          break;
        }
      }
      const int x_row = it.b_row + (int)rank * cta_rows;
      for (int ch = it.c0; ch < it.c1; ++ch) {
        if (!mbar_wait_warp<100>(&stage_free[st], ph ^ 1u, lim, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t* xs = smem_gen + st * S::STAGE_BYTES;
        if (elect_one()) {
          if (codes) {
            uint8_t* cs = xs + S::X_BYTES;
            uint8_t* ss = cs + S::CODE_BYTES;
            if (live) {
              mbar_arrive_expect_tx(&code_full[st], S::CODE_BYTES + gpc * 256);
              tma_load_2d(&maps.codes[it.cls][0], &code_full[st], cs, ch * (BK / 2), y);
              if (mats2)
                tma_load_2d(&maps.codes[it.cls][1], &code_full[st], cs + S::CODE_BYTES / 2, ch * (BK / 2), y);
              tma_load_2d(&maps.scales[it.cls][0], &code_full[st], ss, f0, ys + ch * gpc);
              if (mats2)
                tma_load_2d(&maps.scales[it.cls][1], &code_full[st], ss + S::SCALE_BYTES / 2, f0, ys + ch * gpc);
            } else {
              mbar_arrive(&code_full[st]);
            }
          } else {
            if (leader)
              mbar_arrive_expect_tx(&x_full[st], CTAS * (half ? S::HALF : S::B_ROWS) * BK * 2);
            const uint32_t xb = PAIR ? mapa_shared(smem_u32(&x_full[st]), 0) : smem_u32(&x_full[st]);
            if ((K & 63) == 0 || (ch + 1) * BK <= K) {  // one copy (each costs the issuing lane some 85 cycles)
              tma_load_3d<PAIR>(&maps.x[it.cls][half], xb, xs, 0, x_row, ch * (BK / 64));
            } else {  // the last chunk of a K that ends inside 64 columns
#pragma unroll 1
              for (int h = 0; h < BK / 64; ++h) {
                uint8_t* dst = xs + h * (half ? S::X_SUB / 2 : S::X_SUB);
                for (int b = 0; b < (half ? 1 : 2); ++b)
                  if (PAIR)
                    tma_load_2d_pair(&maps.xt[it.cls], xb, dst + b * S::HALF * 128, ch * BK + h * 64,
                                     x_row + b * S::HALF);
                  else
                    tma_load_2d(&maps.xt[it.cls], &x_full[st], dst + b * S::HALF * 128, ch * BK + h * 64,
                                x_row + b * S::HALF);
              }
            }
          }
        }
        __syncwarp();
        ++used;
        if (PAIR) halves = (halves & ~(1u << st)) | ((uint32_t)half << st);
        if (++st == STAGES) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok) {
      give_up();
    }
    // every issued copy lands before the CTA may exit: the last use of stage i was its fill
    // number (used - 1 - i) / STAGES. (PAIR: the leader's barriers count both CTAs' rows,
    // and the peer waits for the leader at the last cluster barrier. Where either CTA gave
    // up, the copies are settled there, with what both have fetched.)
    if (PAIR && !codes && lane == 0) {
      x_used_s[0] = used;
      x_used_s[1] = (int)halves;
    }
    if (lane == 0 && (codes || leader))
      for (int i = 0; i < STAGES && i < used; ++i) {
        const volatile int never = 0;
        if (!mbar_wait(codes ? &code_full[i] : &x_full[i], (uint32_t)((used - 1 - i) / STAGES) & 1u,
                       WT_DRAIN_LIMIT_NS, PAIR && !codes ? abort_flag : &never)) {
          give_up();
        }
      }
  } else if (warp == 1 || warp == 3) {
    // ---------------------------------------------------------------- matrix issuers
    constexpr int IS = S::ISSUERS;
    const int me = warp >> 1;  // the chunks n (counted over all pieces) with n % IS == me are this issuer's
    if (leader && me < IS) {
      int st = me, as = me, acc = 0, n0 = 0;
      uint32_t ph = 0, accph = 0;
      while (ok && walk.next(it)) {
        if (!mbar_wait_warp(&acc_free[acc], accph ^ 1u, lim, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * S::ACC_COLS + me * BN);
        const int n_inst = (it.rows + 15) & ~15;
        const uint32_t idesc = idesc_bf16(128 * CTAS, n_inst);
        const uint32_t sub = (n_inst / CTAS <= S::HALF ? S::X_SUB / 2 : S::X_SUB) >> 4;  // 64 columns further
        const int first = it.c0 + (IS == 2 && (n0 & 1) != me ? 1 : 0);
        n0 += it.c1 - it.c0;
#pragma unroll 1
        for (int ch = first; ch < it.c1; ch += IS) {
          if (!mbar_wait_warp2(&x_full[st], &a_full[st], ph, lim, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t bd = sdesc_sw128(smem_base + st * S::STAGE_BYTES);
            const uint32_t a = tmem + (uint32_t)(S::NUM_ACC * S::ACC_COLS + as * S::A_COLS);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              umma_ts<PAIR>(d, a + 8 * kk, bd + (kk >> 2) * sub + 2 * (kk & 3), idesc,
                            kk > 0 ? 1u : (uint32_t)(ch > first));
            umma_commit_all<PAIR>(&stage_free[st]);
          }
          __syncwarp();
          as += IS;
          if (as >= A_SLOTS) as -= A_SLOTS;
          st += IS;
          if (st >= STAGES) {
            st -= STAGES;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit_all<PAIR>(&acc_full[acc]);
        __syncwarp();
        if (++acc == S::NUM_ACC) {
          acc = 0;
          accph ^= 1u;
        }
      }
      if (!ok) {
        give_up();
      }
      if (elect_one()) {
        if (PAIR)
          umma_commit_pair(smem_u32(&drain_bar));
        else
          umma_commit(&drain_bar);
        const volatile int never = 0;
        if (!mbar_wait(&drain_bar, 0, WT_DRAIN_LIMIT_NS, &never)) set_status(p.status, MOE_ERR_TIMEOUT);
      }
    }
  } else if (warp >= WT_EXPAND_WARP && warp < S::EPI_WARP) {
    // ---------------------------------------------------------------- expanders
    const int team = (warp - WT_EXPAND_WARP) >> 2, q = warp & 3;
    // (set for each piece: SwiGLU's first product stages two matrices)
    uint32_t code_off, sw, scale_off, scale_pitch;
    const int gl2 = 31 - __clz(p.group);
    auto layout = [&](const bool mats2) {
      const int row = mats2 ? (lane >> 4) * 64 + q * 16 + (lane & 15) : q * 32 + lane;  // of the staged codes
      code_off = S::X_BYTES + row * (BK / 2);
      sw = BK == 256 ? row & 7 : (row >> 1) & 3;  // the TMA's 128- or 64-byte swizzle
      // scales: [matrix][group][64 rows] or [group][128 rows]
      scale_off = S::X_BYTES + S::CODE_BYTES +
                  (mats2 ? (lane >> 4) * (S::SCALE_BYTES / 2) + (q * 16 + (lane & 15)) * 2 : row * 2);
      scale_pitch = mats2 ? 128 : 256;
    };
    layout(wt_cta_f<BN, EPI>(0) == 64);
    const uint32_t t_lane = tmem + ((uint32_t)(q * 32) << 16) + S::NUM_ACC * S::ACC_COLS;
    int st = 0, as = 0, turn = 0;
    uint32_t ph = 0;
    // (before the first such chunk the wait passes at once)
    auto slot_free = [&]() {
      const bool wrap = st < A_SLOTS;
      return mbar_wait_warp(&stage_free[wrap ? st - A_SLOTS + STAGES : st - A_SLOTS], ph ^ (wrap ? 1u : 0u), lim,
                            abort_flag);
    };
    bool dry = true;  // the first turn, before there is work
    it.cls = 0;
    it.c0 = 0;
    it.c1 = 1;
    int ng = 0;
    do {
#pragma unroll 1
      for (int ch = it.c0; ch < it.c1; ++ch) {
        if (dry || turn == team) {
          if (!dry && !mbar_wait_warp(&code_full[st], ph, lim, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t base = smem_base + st * S::STAGE_BYTES;
          // the codes of a short chunk are fetched before the wait for its slot, those of a
          // long one 64 columns at a time (all of them held at once slowed the unpacking)
          constexpr bool EARLY = BK == 128;
          uint4 cw[BK / 32];
          uint32_t sc[BK / 32];
          bool few = true;
#pragma unroll
          for (int i = 0; i < BK / 32; ++i) {
            const int gi = (i * 32) >> gl2;
            if (EARLY) cw[i] = lds128(base + code_off + ((i ^ sw) << 4));
            if (i > 0 && ((i * 32) & (p.group - 1))) {  // the same group as the granule before
              sc[i] = sc[i > 0 ? i - 1 : 0];
              continue;
            }
            sc[i] = lds16(base + scale_off + gi * scale_pitch);
            if (ch * (BK >> gl2) + gi >= ng) sc[i] = 0u;  // behind K: x is zero there, the scale not this row's
            few = few && w4_scale_is_short(sc[i]);
          }
          few = __all_sync(0xffffffffu, few);
          if (!dry && !slot_free()) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t t_slot = t_lane + as * S::A_COLS;
#pragma unroll
          for (int h = 0; h < BK / 64; ++h) {  // 64 columns at a time
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 c4 = EARLY ? cw[2 * h + i] : lds128(base + code_off + (((2 * h + i) ^ sw) << 4));
              const uint32_t w[4] = {c4.x, c4.y, c4.z, c4.w};
              const uint32_t ss = few ? sc[2 * h + i] * 0x10001u : 0x3F803F80u, ms = mul_bf16x2(ss, 0xC1C0C1C0u);
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i * 16 + j * 4 + e] = w4_pair_scaled(w[j], e, ss, ms);
            }
            if (!few) {
              // A scale of another origin, or a large one: code - 8 (exact) came out above.
              // Codes behind K, in a short last group, read as -8, which such a scale may
              // take to infinity: zero. (K is a multiple of the 32 columns of a granule.)
              const int left = p.cls[it.cls].K - ch * BK - 64 * h;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                v[k] = mul_bf16x2(v[k], 32 * (k >> 4) < left ? sc[2 * h + (k >> 4)] * 0x10001u : 0u);
            }
            tmem_st_x32(t_slot + h * 32, v);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          // (relaxed: the stores to tensor memory have completed, and a release at
          // cluster scope would wait for much more)
          if (lane == 0 && !dry) {
            if (leader)
              mbar_arrive_relaxed(&a_full[st]);
            else
              mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&a_full[st]), 0));
          }
        }
        if (dry) break;
        if (++turn == S::TEAMS) turn = 0;
        if (++as == A_SLOTS) as = 0;
        if (++st == STAGES) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (dry) {
        dry = false;
        __syncthreads();  // the schedule is there
      }
      if (!ok || !walk.next(it)) break;
      if (TWO) layout(wt_cta_f<BN, EPI>(it.cls >> 1) == 64);
      ng = (p.cls[it.cls].K + p.group - 1) >> gl2;
    } while (true);
    if (!ok) {
      give_up();
    }
  } else if (warp >= S::EPI_WARP) {
    // ---------------------------------------------------------------- epilogue
    // (the EW / 4 warps of a lane quarter take alternate chunks of 16 rows)
    const int q = warp & 3, ew = warp - S::EPI_WARP;
    const int cfirst = 16 * (ew >> 2);
    constexpr int CSTEP = 16 * (EW / 4);
    int acc = 0, n0 = 0;
    uint32_t accph = 0;
    bool left_first = !TWO;
    auto leave_first = [&]() {  // once a launch, by every epilogue warp, whatever happened before
      left_first = true;
      __threadfence();
      asm volatile("fence.proxy.async.global;" ::: "memory");
      __syncwarp();
      if (lane == 0) atomicAdd(p.grid_count, blockIdx.x || ew ? 1ull : W4_COUNT - (gridDim.x * EW - 1));
    };
    while (ok && walk.next(it)) {
      const W4Class& c = p.cls[it.cls];
      const int phase = EPI == EPI_DOWN ? 1 : it.cls >> 1;
      if (TWO && phase == 1 && !left_first) leave_first();
      const int f0 = (it.mt * CTAS + (int)rank) * (EPI == EPI_DOWN ? 128 : wt_cta_f<BN, EPI>(phase));
      const int rows = it.rows;
      // 16 rows' sums of this lane's weight row -> output rows [c0, c0 + 16)
      auto emit = [&](const int c0, const float (&v)[16]) {
        const int jn = min(16, rows - c0);
        if (EPI == EPI_DOWN || (TWO && phase == 1)) {
          const int feat = f0 + q * 32 + lane;
          const long long r0 = it.out_row + c0;
          float wv = 1.f;
          if (lane < jn) {
            if (c.row_w) {
              wv = c.row_w[r0 + lane];
            } else if (c.task_w) {
              const int qk = c.perm[r0 + lane];
              wv = qk >= 0 && qk < c.max_row ? c.task_w[qk] : 0.f;
            }
          }
          float* o = reinterpret_cast<float*>(c.out) + r0 * c.R + feat;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float w = __shfl_sync(0xffffffffu, wv, j);
            if (j < jn && feat < c.R) o[(long long)j * c.R] = v[j] * w;
          }
        } else if (EPI == EPI_SWIGLU) {
          // lanes 0..15 hold the gate sums of 16 features, lanes 16..31 their up sums: the
          // lower half takes the even rows, the upper half the odd ones
          const bool up = lane >= 16;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * j] : v[2 * j + 1], 16);
            const float g = up ? got : v[2 * j], u = up ? v[2 * j + 1] : got;
            // h is rounded to bf16: it is the next product's tensor-core operand
            stg[ew][2 * j + up][lane & 15] = __float2bfloat16_rn(__fdividef(g, 1.f + __expf(-g)) * u);
          }
          __syncwarp();
          const int j = lane >> 1, f = f0 + q * 16 + (lane & 1) * 8;
          if (j < jn && f < c.R)
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(c.out) + (long long)(it.out_row + c0 + j) * c.R +
                                      f) = *reinterpret_cast<const uint4*>(&stg[ew][j][(lane & 1) * 8]);
          __syncwarp();
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) stg[ew][j][lane] = __float2bfloat16_rn(v[j] < 0.f ? 0.f : v[j]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = (lane >> 2) + 8 * i, f = f0 + q * 32 + (lane & 3) * 8;
            if (j < jn && f < c.R)
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(c.out) +
                                        (long long)(it.out_row + c0 + j) * c.R + f) =
                  *reinterpret_cast<const uint4*>(&stg[ew][j][(lane & 3) * 8]);
          }
          __syncwarp();
        }
      };
      const bool whole = it.wa == it.wb;
      // this warp's part of a walker's partial sums: [row][128 lanes]
      auto part_of = [&](const int w, const int slot) {
        return p.partial + (TWO && phase == 1 ? w4_partial_floats(BN) : 0) +
               ((((size_t)w * 2 + slot) * CTAS + rank) * BN) * 128 + q * 32 + lane;
      };
      float* mine = whole ? nullptr : part_of(walker, it.wa < walker ? 0 : 1);
      if (!mbar_wait_warp<100>(&acc_full[acc], accph, lim, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * S::ACC_COLS);
      auto use = [&](const int c0, const uint32_t (&r)[16]) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
        if (whole) {
          emit(c0, v);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) __stcg(mine + (c0 + j) * 128, v[j]);
        }
        __syncwarp();
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            mbar_arrive_relaxed(&acc_free[acc]);
          else
            mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_free[acc]), 0));
        }
      };
      uint32_t ra[16], rb[16];
      if (S::ISSUERS == 2) {
        // the sum of the issuers' sums; one of them has none when the piece is one chunk
        const int chunks = it.c1 - it.c0;
        const bool both = chunks > 1;
        const uint32_t t_one = t_row + (!both && (n0 & 1) ? BN : 0);
        n0 += chunks;
#pragma unroll 1
        for (int c0 = cfirst; c0 < rows; c0 += CSTEP) {
          tmem_ld_x16(t_one + c0, ra);
          if (both) {
            tmem_ld_x16(t_row + BN + c0, rb);
            tmem_ld_wait_keep(ra, rb);
#pragma unroll
            for (int j = 0; j < 16; ++j) ra[j] = __float_as_uint(__uint_as_float(ra[j]) + __uint_as_float(rb[j]));
          } else {
            tmem_ld_wait_keep(ra);
          }
          if (c0 + CSTEP >= rows) release();
          use(c0, ra);
        }
        if (cfirst >= rows) release();
      } else {
        // the loads of one 16-column chunk are in flight while the one before is used
        if (cfirst < rows) tmem_ld_x16(t_row + cfirst, ra); else release();
#pragma unroll 1
        for (int c0 = cfirst; c0 < rows; c0 += 2 * CSTEP) {
          tmem_ld_wait_keep(ra);
          if (c0 + CSTEP < rows) tmem_ld_x16(t_row + c0 + CSTEP, rb); else release();
          use(c0, ra);
          if (c0 + CSTEP >= rows) break;
          tmem_ld_wait_keep(rb);
          if (c0 + 2 * CSTEP < rows) tmem_ld_x16(t_row + c0 + 2 * CSTEP, ra); else release();
          use(c0 + CSTEP, rb);
        }
      }
      if (++acc == S::NUM_ACC) {
        acc = 0;
        accph ^= 1u;
      }
      if (!whole) {
        // the last of the tile's walkers to get here adds the parts, in the order of K
        __threadfence();
        __syncwarp();
        unsigned* const counter = p.counters + (TWO ? (2 * (int)(launch_s & 1) + phase) * W4_COUNTERS2 : 0) +
                                  (it.wa * CTAS + (int)rank) * EW + ew;
        unsigned n = 0;
        if (lane == 0) n = atomicAdd(counter, 1u);
        n = __shfl_sync(0xffffffffu, n, 0);
        if (n == (unsigned)(it.wb - it.wa)) {
          if (!TWO && lane == 0) *counter = 0u;  // whether a launch of the other product follows or not
          __threadfence();
#pragma unroll 1
          for (int c0 = cfirst; c0 < rows; c0 += CSTEP) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.f;
#pragma unroll 2
            for (int w = it.wa; w <= it.wb; ++w) {
              const float* o = part_of(w, w == it.wa ? 1 : 0) + c0 * 128;
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] += __ldcg(o + j * 128);
            }
            emit(c0, v);
          }
        }
      }
    }
    if (!left_first) leave_first();
    if (!ok) {
      give_up();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (PAIR) {
    cluster_sync_all();  // neither CTA leaves while the other may signal it or read its memory
    if (__builtin_expect(settle_s, 0)) {  // (alike in both CTAs)
      if (leader && warp == 2 && lane == 0)
        wt_settle<STAGES>(x_full, x_used_s, S::HALF * BK * 2, S::B_ROWS * BK * 2);
      __syncwarp();
      cluster_sync_all();  // both CTAs' rows have landed
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_g<PAIR>(tmem, 512);
  }
}

bool make_map_2d(CUtensorMap* m, const void* ptr, CUtensorMapDataType type, long long inner, long long rows,
                 long long pitch, int box_inner, int box_rows, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc || !ptr || inner <= 0 || rows <= 0 || pitch % 16) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return enc(m, type, 2, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 rows [rows, K] as [K / 64][rows][64]: one copy brings `subs` groups of 64 columns
// of box_rows rows, each group with the 128-byte swizzle of a K-major operand.
bool make_map_rows(CUtensorMap* m, const void* ptr, long long K, long long rows, int box_rows, int subs) {
  EncodeTiledFn enc = encode_fn();
  if (!enc || !ptr || K <= 0 || rows <= 0 || K % 8) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)std::max(1LL, K / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)K * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)subs}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int EPI>
cudaError_t launch_impl(const W4Params& p, cudaStream_t s) {
  using S = WtShape<BN>;
  WtMaps<S::PHASES> maps;
  for (int i = 0; i < 2 * S::PHASES; ++i) {
    const W4Class& c = p.cls[i % 2 < p.n_classes ? i : i & ~1];
    const bool mats2 = EPI == EPI_SWIGLU && i < 2;
    const int ng = (c.K + p.group - 1) / p.group, rows = mats2 ? 64 : 128;
    for (int j = 0; j < 2; ++j) {
      const W4Matrix& a = mats2 && j ? c.a1 : c.a0;
      if (!make_map_2d(&maps.codes[i][j], a.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.K / 2, (long long)c.n_groups * c.R,
                       c.K / 2, S::BK / 2, rows,
                       S::BK == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
          !make_map_2d(&maps.scales[i][j], a.scales, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, c.R, (long long)c.n_groups * ng,
                       2LL * c.R, rows, S::BK / p.group, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    }
    if (!make_map_2d(&maps.xt[i], c.b, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, c.K, c.b_rows, 2LL * c.K, 64, S::HALF,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_rows(&maps.x[i][0], c.b, c.K, c.b_rows, S::B_ROWS, S::BK / 64) ||
        !make_map_rows(&maps.x[i][1], c.b, c.K, c.b_rows, S::HALF, S::BK / 64))
      return cudaErrorInvalidValue;
  }
  auto kern = w4_gemm_kernel<BN, EPI>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::THREADS);
  cfg.dynamicSmemBytes = S::DYN_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  int attrs = 1;
  if (S::PAIR) {
    attr[attrs].id = cudaLaunchAttributeClusterDimension;
    attr[attrs].val.clusterDim.x = 2;
    attr[attrs].val.clusterDim.y = 1;
    attr[attrs].val.clusterDim.z = 1;
    ++attrs;
  }
  if (S::PHASES == 2) {
    attr[attrs].id = cudaLaunchAttributeCooperative;
    attr[attrs].val.cooperative = 1;
    ++attrs;
  }
  static int walkers[64] = {0};  // a device: CTAs or pairs that can be resident at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!walkers[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::DYN_SMEM);
    if (e != cudaSuccess) return e;
    int n = num_sms();
    if (S::PAIR) {
      cfg.gridDim = dim3(num_sms() & ~1);
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;  // the occupancy query takes the cluster shape alone
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
    }
    walkers[dev] = std::max(1, std::min(n, W4_MAX_CTAS / (S::PAIR ? 2 : 1)));
  }
  cfg.gridDim = dim3(walkers[dev] * (S::PAIR ? 2 : 1));
  cfg.attrs = attr;
  cfg.numAttrs = attrs;
  e = cudaLaunchKernelEx(&cfg, kern, maps, p);
  count_launch();
  return e;
}

}  // namespace

// Input rows a tile: enough for most segments to be one tile (every further tile of a
// segment expands the expert's weights again), no more than that (a stage's bytes, and
// the tensor memory left for expanded weights). avg_rows is the routed experts' mean alone;
// the shared experts' segments of T rows take the same tiles, and where those are short
// their weights are expanded often: 1000 tokens, one of 128 experts each (2048 x 1408), run
// 207 us, with two shared experts 338 (16-row tiles, 63 a shared expert); six of 64 experts
// each 210 and 243.
int w4_pick_bn(long long T, double avg_rows) {
  const double want = std::min((double)T, 2.0 * avg_rows);
  return want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : std::min((double)T, avg_rows) <= 160 ? 128 : 192;
}

// (at 64 rows 96 tokens on 8 experts of 4096 x 4096 ran 107 us in two launches, 102 in one;
// at 128 rows 506 tokens on 8 of 4096 x 14336 ran 372 and 380.)
bool w4_both_products(int bn) { return bn <= 64; }

int w4_grid_kind(int bn) { return bn <= 32 ? 0 : 1; }

// Long segments' tiles: 224 rows with one sum in tensor memory where every tile runs over
// at least 32 chunks of K, 192 rows with two otherwise (8 experts of 4096 x 14336, 4096
// tokens: up 1350 -> 1279 us, down 697 -> 671; at K = 1408 down 103 -> 126, so not there).
static bool w4_deep(const W4Params& p) {
  for (int i = 0; i < p.n_classes; ++i)
    if (p.cls[i].K < 4096) return false;
  return true;
}

size_t w4_partial_bytes(int bn) { return w4_partial_floats(bn == 192 ? 224 : bn) * sizeof(float) * (w4_both_products(bn) ? 2 : 1); }

cudaError_t launch_w4_gemm(int epi, int bn, const W4Params& p, cudaStream_t s) {
  if (bn == 192 && w4_deep(p)) bn = 224;
#define MOE_W4_CASE(BN_)                                                  \
  if (bn == BN_) {                                                        \
    static_assert(WtShape<BN_>::PHASES == (BN_ <= 64 ? 2 : 1), "phases"); \
    if (epi == EPI_SWIGLU) return launch_impl<BN_, EPI_SWIGLU>(p, s);     \
    if (epi == EPI_RELU) return launch_impl<BN_, EPI_RELU>(p, s);         \
  }
  MOE_W4_CASE(16)
  MOE_W4_CASE(32)
  MOE_W4_CASE(64)
  MOE_W4_CASE(128)
  MOE_W4_CASE(192)
  MOE_W4_CASE(224)
#undef MOE_W4_CASE
  if (epi == EPI_DOWN && bn == 128) return launch_impl<128, EPI_DOWN>(p, s);
  if (epi == EPI_DOWN && bn == 192) return launch_impl<192, EPI_DOWN>(p, s);
  if (epi == EPI_DOWN && bn == 224) return launch_impl<224, EPI_DOWN>(p, s);
  return cudaErrorInvalidValue;
}

// Turns of a block: all of them where that still gives every SM several blocks, else one
// (a small matrix is bound by one block's latency).
static int quantizer_turns(long long n, int rows, int cols) {
  const long long blocks = n * ((cols + QW_COLS - 1) / QW_COLS) * ((rows + QW_ROWS - 1) / QW_ROWS);
  return blocks >= 16LL * QW_TURNS * num_sms() ? QW_TURNS : 1;
}

cudaError_t launch_quantize_w4(long long n, int rows, int cols, int group, const void* src, uint8_t* codes,
                               void* scales, cudaStream_t s) {
  const int turns = quantizer_turns(n, rows, cols), block_rows = QW_ROWS * turns;
  const dim3 grid((cols + QW_COLS - 1) / QW_COLS, (rows + block_rows - 1) / block_rows, (unsigned)n);
  auto kern = group == 32 ? quantize_w4_kernel<32> : group == 64 ? quantize_w4_kernel<64> : quantize_w4_kernel<128>;
  cudaError_t e = launch_k(kern, grid, dim3(QW_WARPS * 32), 0, s, rows, cols, turns, (const uint4*)src, (uint32_t*)codes,
                           (__nv_bfloat16*)scales);
  count_launch();
  return e;
}

cudaError_t launch_dequantize_w4(long long n, int rows, int cols, int group, const uint8_t* codes, const void* scales,
                                 void* dst, cudaStream_t s) {
  const int turns = quantizer_turns(n, rows, cols), block_rows = QW_ROWS * turns;
  const dim3 grid((cols + QW_COLS - 1) / QW_COLS, (rows + block_rows - 1) / block_rows, (unsigned)n);
  auto kern =
      group == 32 ? dequantize_w4_kernel<32> : group == 64 ? dequantize_w4_kernel<64> : dequantize_w4_kernel<128>;
  cudaError_t e = launch_k(kern, grid, dim3(QW_WARPS * 32), 0, s, rows, cols, turns, (const uint32_t*)codes,
                           (const uint16_t*)scales, (uint4*)dst);
  count_launch();
  return e;
}

}  // namespace moe
