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

#include "w4.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------------ quantizer
constexpr int QW_WARPS = 8;    // warps a block
constexpr int QW_ROWS = 32;    // rows a block, 4 a warp
constexpr int QW_COLS = 256;   // columns a block: 8 a lane

__device__ __forceinline__ float scale_5bits(float amax) {
  uint32_t u = __float_as_uint(__fdiv_rn(amax, 7.f));
  u = (u + 0x3FFFFu + ((u >> 19) & 1u)) & 0xFFF80000u;  // nearest, ties to even, at mantissa bit 19
  return u >= 0x00800000u ? __uint_as_float(u) : 1.f;
}

// Code + 8 of v: a saturating integer conversion, so any input gives a code.
__device__ __forceinline__ uint32_t code4(float v, float sc) {
  return (uint32_t)(min(7, max(-8, __float2int_rn(__fdiv_rn(v, sc)))) + 8);
}

// A block takes QW_ROWS rows x QW_COLS columns: a lane 8 columns of 4 rows. The group's
// maximum comes from the G / 8 lanes that share it; the scales meet in shared memory so
// that each group's QW_ROWS scales leave as one 64-byte run of the group-major layout.
template <int G>
__global__ void __launch_bounds__(QW_WARPS * 32)
    quantize_w4_kernel(int rows, int cols, const uint4* __restrict__ src, uint32_t* __restrict__ codes,
                       __nv_bfloat16* __restrict__ scales) {
  constexpr int GPB = QW_COLS / G;
  __shared__ __nv_bfloat16 sc_s[GPB][QW_ROWS];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long mat = blockIdx.z;
  const int ng = (cols + G - 1) / G;
  const int c8 = blockIdx.x * (QW_COLS / 8) + lane, n8 = cols >> 3;
  const int row0 = blockIdx.y * QW_ROWS + warp * 4;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c8 < n8 && row0 + i < rows) v[i] = src[(mat * rows + row0 + i) * n8 + c8];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    float f[8], amax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      amax = fmaxf(amax, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
    }
#pragma unroll
    for (int off = G / 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const float sc = scale_5bits(amax);
    uint32_t word = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) word |= (code4(f[2 * j], sc) << (4 * j)) | (code4(f[2 * j + 1], sc) << (16 + 4 * j));
    if (c8 < n8 && row0 + i < rows) codes[(mat * rows + row0 + i) * n8 + c8] = word;
    if (lane % (G / 8) == 0) sc_s[lane / (G / 8)][warp * 4 + i] = __float2bfloat16_rn(sc);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < GPB * QW_ROWS; i += QW_WARPS * 32) {
    const int g = blockIdx.x * GPB + i / QW_ROWS, row = blockIdx.y * QW_ROWS + i % QW_ROWS;
    if (g < ng && row < rows) scales[(mat * ng + g) * rows + row] = sc_s[i / QW_ROWS][i % QW_ROWS];
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

// The inverse: bf16(code * scale) (exact for the quantizer's scales). A lane turns one
// word (8 columns) of 4 neighbouring rows into 16 bytes each.
template <int G>
__global__ void __launch_bounds__(QW_WARPS * 32)
    dequantize_w4_kernel(int rows, int cols, const uint32_t* __restrict__ codes,
                         const uint16_t* __restrict__ scales, uint4* __restrict__ dst) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long mat = blockIdx.z;
  const int ng = (cols + G - 1) / G;
  const int c8 = blockIdx.x * (QW_COLS / 8) + lane, n8 = cols >> 3;
  const int row0 = blockIdx.y * QW_ROWS + warp * 4;
  if (c8 >= n8 || row0 >= rows) return;  // rows % 8 == 0: the 4 rows exist together
  const uint2 s4 = *reinterpret_cast<const uint2*>(scales + (mat * ng + 8 * c8 / G) * rows + row0);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = codes[(mat * rows + row0 + i) * n8 + c8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = ((i & 2) ? s4.y : s4.x) >> (16 * (i & 1)) & 0xFFFFu, ss = h | (h << 16);
    uint4 o;
    o.x = mul_bf16x2(w4_pair(w[i]), ss);
    o.y = mul_bf16x2(w4_pair(w[i] >> 4), ss);
    o.z = mul_bf16x2(w4_pair(w[i] >> 8), ss);
    o.w = mul_bf16x2(w4_pair(w[i] >> 12), ss);
    dst[(mat * rows + row0 + i) * n8 + c8] = o;
  }
}

// ------------------------------------------------------------------ products over short segments
// y = x . W^T for a few rows of x per expert, where the codes' bytes are what counts.
//
// A block of 16 warps takes a unit: a block of weight rows of one matrix (or of the gate
// and up matrices together) and a tile of at most 8 NT input rows, over the whole
// reduction length. A warp holds 32 weight rows (16 of gate and 16 of up, or 32 of down)
// and every KW-th chunk of 128 columns; the KW warps' sums meet in shared memory. The
// codes stream through a ring of STAGES chunks a warp filled by 16-byte asynchronous
// copies, which runs on across units, so the loads of the next unit are in flight while
// this one is summed up. In registers a word becomes four bf16 pairs (code - 8, exact)
// for mma.m16n8k16 with the input rows as the N side; the fp32 sum of a group is then
// multiplied by the group's scale in fp32, so no weight is rounded. (The matrix unit of
// this kernel is the warp-level one: with N = 8..32 it is far from its rate, operands
// come straight from the registers that unpack them, and no wait between warps is
// needed; long segments go to the tcgen05 kernel.)
//
// A lane (g = lane / 4, t = lane % 4) takes the word t of each 32-column granule for the
// rows g and g + 8, and 16 bytes of input row g at the same columns: the four pairs of a
// word are the k pairs of two products on both sides.
constexpr int SG_WARPS = 16;
constexpr int SG_CHUNK = 128;                   // columns a stage
constexpr int SG_STAGES = 4;
constexpr int SG_CODE_BYTES = 2 * 16 * 64;      // two 16-row tiles x 64 bytes
constexpr int SG_STAGE_BYTES = SG_CODE_BYTES + 2 * 4 * 32;  // and up to 4 groups' scales of each tile's rows
constexpr int SG_MAX_GROUPS = 1040;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return bf16_bits_to_f32(v);
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Active groups in order: gid[pos], its first unit, rows and first input row.
struct SgSched {
  int start[SG_MAX_GROUPS + 1];
  int gid[SG_MAX_GROUPS], rows[SG_MAX_GROUPS], brow[SG_MAX_GROUPS];
  int n;
};

struct SgUnit {
  int cls, g, row0, tok0, ntok, brow;  // weight row of the block, input rows tok0.. (brow: of the segment)
};

template <int NT>
__device__ __forceinline__ SgUnit sg_unit(const W4Params& p, const SgSched& s, int& pos, int u, int rpu) {
  while (s.start[pos + 1] <= u) ++pos;
  SgUnit r;
  const int gi = s.gid[pos], G0 = p.cls[0].n_groups;
  r.cls = gi < G0 ? 0 : 1;
  r.g = gi - (r.cls ? G0 : 0);
  const int tiles = (s.rows[pos] + 8 * NT - 1) / (8 * NT), local = u - s.start[pos];
  r.tok0 = (local % tiles) * 8 * NT;  // a block of weights meets all its input tiles in a row (L2)
  r.row0 = (local / tiles) * rpu;
  r.ntok = min(8 * NT, s.rows[pos] - r.tok0);
  r.brow = s.brow[pos];
  return r;
}

template <int NT, int MATS, int EPI>
__global__ void __launch_bounds__(SG_WARPS * 32, 1) w4_stream_kernel(const __grid_constant__ W4Params p, int kw_log2) {
  constexpr int TILE_ROWS = MATS == 2 ? 16 : 32;  // output features a warp
  constexpr int NBUF = NT <= 2 ? 2 : 1;           // buffers of partial sums
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ SgSched sched;
  uint8_t* ring_gen = dyn;
  float* part = reinterpret_cast<float*>(dyn + SG_WARPS * SG_STAGES * SG_STAGE_BYTES);  // [NBUF][warp][8 NT][32]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KW = 1 << kw_log2, RW = SG_WARPS >> kw_log2;
  const int rw = warp >> kw_log2, kw = warp & (KW - 1);
  const int rpu = RW * TILE_ROWS;  // output features a unit
  const int G0 = p.cls[0].n_groups, G = G0 + (p.n_classes > 1 ? p.cls[1].n_groups : 0);
  pdl_launch_dependents();
  pdl_wait();
  if (warp == 0) {  // the units of every group with rows: a prefix sum over 32 runs of groups
    const int per = (G + 31) / 32, lo = lane * per, hi = min(G, lo + per);
    int n = 0, units = 0;
    auto seg = [&](int gi, int& rows, int& brow) {
      const int cl = gi < G0 ? 0 : 1, g = gi - (cl ? G0 : 0);
      const W4Class& c = p.cls[cl];
      if (c.seg_off) {
        const int a = c.seg_off[g], b = c.seg_off[g + 1];
        const bool bad = a < 0 || b < a || b > c.max_row;
        if (bad) set_status(p.status, MOE_ERR_DEVICE_INDEX);
        rows = bad ? 0 : b - a;
        brow = bad ? 0 : a;
      } else {
        rows = c.const_rows;
        brow = g * c.b_group_stride;
      }
      return ((rows + 8 * NT - 1) / (8 * NT)) * ((c.R + rpu - 1) / rpu);
    };
    for (int gi = lo; gi < hi; ++gi) {
      int rows, brow;
      const int k = seg(gi, rows, brow);
      units += k;
      n += k > 0;
    }
    int in = n, iu = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, in, off), b = __shfl_up_sync(0xffffffffu, iu, off);
      if (lane >= off) {
        in += a;
        iu += b;
      }
    }
    int pos = in - n, u = iu - units;
    for (int gi = lo; gi < hi; ++gi) {
      int rows, brow;
      const int k = seg(gi, rows, brow);
      if (!k) continue;
      sched.start[pos] = u;
      sched.gid[pos] = gi;
      sched.rows[pos] = rows;
      sched.brow[pos] = brow;
      ++pos;
      u += k;
    }
    if (lane == 31) {
      // an earlier kernel of the layer flagged a device error: its tables are not used
      const int prior = p.status ? *reinterpret_cast<volatile int*>(p.status) : 0;
      sched.n = prior ? 0 : in;
      sched.start[in] = iu;
    }
  }
  __syncthreads();
  const int total = sched.n ? sched.start[sched.n] : 0;
  const int gpc = SG_CHUNK / p.group;  // groups a chunk
  const uint32_t ring = smem_u32(ring_gen) + warp * SG_STAGES * SG_STAGE_BYTES;

  // ---- producer state: the next chunk this warp loads
  int pu = blockIdx.x, ppos = 0, pc = kw, pnc = 0, slot_in = 0;
  SgUnit pun;
  bool have = false;
  auto issue = [&]() {
    while (pu < total) {
      if (!have) {
        pun = sg_unit<NT>(p, sched, ppos, pu, rpu);
        pnc = (p.cls[pun.cls].K + SG_CHUNK - 1) / SG_CHUNK;
        pc = kw;
        have = true;
      }
      if (pc < pnc) break;
      have = false;
      pu += gridDim.x;
    }
    if (pu < total) {
      const W4Class& c = p.cls[pun.cls];
      const uint32_t st = ring + slot_in * SG_STAGE_BYTES;
      const int row0 = pun.row0 + rw * TILE_ROWS, kb = c.K >> 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int id = i * 32 + lane, tile = id >> 6, r = (id >> 2) & 15, gr = id & 3;
        const int byte = pc * (SG_CHUNK / 2) + gr * 16;
        const uint8_t* base = MATS == 2 && tile ? c.a1.codes : c.a0.codes;
        const int row = min(row0 + (MATS == 2 ? 0 : tile * 16) + r, c.R - 1);  // rows past the matrix: not stored
        if (byte < kb)
          cp_async16(st + tile * 1024 + r * 64 + ((gr ^ ((r >> 1) & 3)) << 4),
                     base + ((size_t)pun.g * c.R + row) * kb + byte);
      }
      if (lane < 4 * gpc) {  // [tile][group][16 rows] scales, two 16-byte halves each
        const int half = lane & 1, tile = (lane >> 1) & 1, q = lane >> 2;
        const int ng = (c.K + p.group - 1) / p.group, grp = pc * gpc + q;
        const __nv_bfloat16* base = MATS == 2 && tile ? c.a1.scales : c.a0.scales;
        const int row = min(row0 + (MATS == 2 ? 0 : tile * 16) + half * 8, c.R - 8);
        if (grp < ng)
          cp_async16(st + SG_CODE_BYTES + (tile * 4 + q) * 32 + half * 16,
                     base + ((size_t)pun.g * ng + grp) * c.R + row);
      }
      pc += KW;
    }
    cp_async_commit();
    if (++slot_in == SG_STAGES) slot_in = 0;
  };
#pragma unroll 1
  for (int i = 0; i < SG_STAGES - 1; ++i) issue();

  const int g8 = lane >> 2, t4 = lane & 3;
  int cpos = 0, slot = 0, buf = 0;
#pragma unroll 1
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const SgUnit un = sg_unit<NT>(p, sched, cpos, u, rpu);
    const W4Class& c = p.cls[un.cls];
    const int nc = (c.K + SG_CHUNK - 1) / SG_CHUNK;
    const int nt_n = (un.ntok + 7) >> 3;
    float tot[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) tot[i][j][e] = 0.f;
    const __nv_bfloat16* xr = c.b + (size_t)(un.brow + un.tok0 + g8) * c.K + t4 * 8;
#pragma unroll 1
    for (int ch = kw; ch < nc; ch += KW) {
      cp_async_wait<SG_STAGES - 2>();
      __syncwarp();
      issue();  // into the slot that was read before the last __syncwarp
      const uint32_t st = ring + slot * SG_STAGE_BYTES;
      if (++slot == SG_STAGES) slot = 0;
      float acc[2][NT][4];
#pragma unroll
      for (int gr = 0; gr < 4; ++gr) {
        const int k = ch * SG_CHUNK + gr * 32;
        if (k >= c.K) break;
        if (((gr * 32) & (p.group - 1)) == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
        }
        uint4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b[j] = make_uint4(0u, 0u, 0u, 0u);
          if (j * 8 + g8 < un.ntok) b[j] = *reinterpret_cast<const uint4*>(xr + (size_t)j * 8 * c.K + k);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a = st + i * 1024 + g8 * 64 + ((gr ^ ((g8 >> 1) & 3)) << 4) + t4 * 4;
          const uint32_t w0 = lds32(a), w1 = lds32(a + 512);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a0 = w4_pair(w0 >> (8 * h)), a1 = w4_pair(w1 >> (8 * h));
            const uint32_t a2 = w4_pair(w0 >> (8 * h + 4)), a3 = w4_pair(w1 >> (8 * h + 4));
#pragma unroll
            for (int j = 0; j < NT; ++j)
              if (j < nt_n) mma_16816(acc[i][j], a0, a1, a2, a3, h ? b[j].z : b[j].x, h ? b[j].w : b[j].y);
          }
        }
        if ((((gr + 1) * 32) & (p.group - 1)) == 0 || k + 32 >= c.K) {  // the group (or the row) ends
          const int q = (gr * 32) / p.group;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a = st + SG_CODE_BYTES + (i * 4 + q) * 32 + g8 * 2;
            const float s0 = lds_bf16(a), s1 = lds_bf16(a + 16);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              tot[i][j][0] = fmaf(acc[i][j][0], s0, tot[i][j][0]);
              tot[i][j][1] = fmaf(acc[i][j][1], s0, tot[i][j][1]);
              tot[i][j][2] = fmaf(acc[i][j][2], s1, tot[i][j][2]);
              tot[i][j][3] = fmaf(acc[i][j][3], s1, tot[i][j][3]);
            }
          }
        }
      }
    }
    // the KW partial sums of each output meet in shared memory, in fragment order
    float* pw = part + ((size_t)buf * SG_WARPS + warp) * (8 * NT * 32) + lane;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) pw[((i * NT + j) * 4 + e) * 32] = tot[i][j][e];
    __syncthreads();
    // frag f = (tile, j, e): one warp-wide run of 32 values a fragment and source warp
    constexpr int FR = 4 * NT * (MATS == 2 ? 1 : 2);  // output fragments a row block
    const float* pb = part + (size_t)buf * SG_WARPS * (8 * NT * 32) + lane;
#pragma unroll 1
    for (int id = warp; id < RW * FR; id += SG_WARPS) {
      const int rb = id / FR, f = id % FR;
      const int tile = MATS == 2 ? 0 : f / (4 * NT), j = (f / 4) % NT, e = f & 3;
      const int tok = j * 8 + 2 * t4 + (e & 1);
      const int feat = un.row0 + rb * TILE_ROWS + tile * 16 + g8 + ((e & 2) ? 8 : 0);
      if (tok >= un.ntok || feat >= c.R) continue;
      const float* q = pb + (size_t)(rb << kw_log2) * (8 * NT * 32);
      float v0 = 0.f, v1 = 0.f;
#pragma unroll 4
      for (int w = 0; w < KW; ++w) {
        v0 += q[(size_t)w * (8 * NT * 32) + f * 32];
        if (MATS == 2) v1 += q[(size_t)w * (8 * NT * 32) + (4 * NT + f) * 32];
      }
      const long long orow =
          (long long)(c.seg_off ? un.brow : un.g * c.out_group_stride) + un.tok0 + tok;
      if (EPI == EPI_DOWN) {
        float wgt = 1.f;
        if (c.row_w) {
          wgt = c.row_w[orow];
        } else if (c.task_w) {
          const int qk = c.perm[orow];
          wgt = qk >= 0 && qk < c.max_row ? c.task_w[qk] : 0.f;
        }
        reinterpret_cast<float*>(c.out)[orow * c.R + feat] = v0 * wgt;
      } else {
        // h is rounded to bf16: it is the next product's tensor-core operand
        const float h = EPI == EPI_SWIGLU ? v0 / (1.f + __expf(-v0)) * v1 : (v0 < 0.f ? 0.f : v0);
        reinterpret_cast<__nv_bfloat16*>(c.out)[orow * c.R + feat] = __float2bfloat16_rn(h);
      }
    }
    if (NBUF == 2)
      buf ^= 1;  // the next write of this buffer is two barriers away
    else
      __syncthreads();
  }
  cp_async_wait<0>();
}

template <int NT, int MATS, int EPI>
cudaError_t launch_stream(const W4Params& p, int kw_log2, cudaStream_t s) {
  constexpr size_t SMEM = SG_WARPS * SG_STAGES * SG_STAGE_BYTES +
                          (NT <= 2 ? 2 : 1) * SG_WARPS * (8 * NT * 32) * sizeof(float);
  auto kern = w4_stream_kernel<NT, MATS, EPI>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
  if (e != cudaSuccess) return e;
  e = launch_k(kern, dim3(num_sms()), dim3(SG_WARPS * 32), SMEM, s, p, kw_log2);
  count_launch();
  return e;
}

// The 16 warps of a block split the reduction KW ways and the rows 16 / KW ways. KW is
// the power of two that leaves the fewest chunk slots unused (chunks of the last round),
// the larger one on a tie: units of fewer rows spread more evenly over the SMs.
int pick_kw_log2(const W4Params& p) {
  int best = 4;
  double best_cost = 1e30;
  for (int l = 4; l >= 1; --l) {
    const int nc = (p.cls[0].K + SG_CHUNK - 1) / SG_CHUNK, kw = 1 << l;
    const double cost = (double)((nc + kw - 1) / kw * kw) / nc;
    if (cost < best_cost - 1e-9) {
      best_cost = cost;
      best = l;
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_w4_gemm(int epi, const W4Params& p, int max_rows, double avg_rows, cudaStream_t s) {
  const int kw = pick_kw_log2(p);
  (void)avg_rows;
#define MOE_W4_STREAM(NT_)                                                                 \
  do {                                                                                     \
    if (epi == EPI_SWIGLU) return launch_stream<NT_, 2, EPI_SWIGLU>(p, kw, s);             \
    if (epi == EPI_RELU) return launch_stream<NT_, 1, EPI_RELU>(p, kw, s);                 \
    if (epi == EPI_DOWN) return launch_stream<NT_, 1, EPI_DOWN>(p, kw, s);                 \
    return cudaErrorInvalidValue;                                                          \
  } while (0)
  if (max_rows <= 8) MOE_W4_STREAM(1);
  if (max_rows <= 16) MOE_W4_STREAM(2);
  MOE_W4_STREAM(4);
#undef MOE_W4_STREAM
}

cudaError_t launch_quantize_w4(long long n, int rows, int cols, int group, const void* src, uint8_t* codes,
                               void* scales, cudaStream_t s) {
  const dim3 grid((cols + QW_COLS - 1) / QW_COLS, (rows + QW_ROWS - 1) / QW_ROWS, (unsigned)n);
  auto kern = group == 32 ? quantize_w4_kernel<32> : group == 64 ? quantize_w4_kernel<64> : quantize_w4_kernel<128>;
  cudaError_t e = launch_k(kern, grid, dim3(QW_WARPS * 32), 0, s, rows, cols, (const uint4*)src, (uint32_t*)codes,
                           (__nv_bfloat16*)scales);
  count_launch();
  return e;
}

cudaError_t launch_dequantize_w4(long long n, int rows, int cols, int group, const uint8_t* codes, const void* scales,
                                 void* dst, cudaStream_t s) {
  const dim3 grid((cols + QW_COLS - 1) / QW_COLS, (rows + QW_ROWS - 1) / QW_ROWS, (unsigned)n);
  auto kern =
      group == 32 ? dequantize_w4_kernel<32> : group == 64 ? dequantize_w4_kernel<64> : dequantize_w4_kernel<128>;
  cudaError_t e = launch_k(kern, grid, dim3(QW_WARPS * 32), 0, s, rows, cols, (const uint32_t*)codes,
                           (const uint16_t*)scales, (uint4*)dst);
  count_launch();
  return e;
}

}  // namespace moe
