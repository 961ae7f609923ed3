// 4-bit expert weights: the internal interface of csrc/w4.cu.
//
// A matrix [R, K] is held as codes [R, K / 2] bytes and bf16 scales [ceil(K / G), R]
// (group-major: the scales of a tile's rows are one run a group, a box of the tensor map
// that fetches them). A row is a sequence of 32-bit words of 8 columns; column 2i of a word sits in bits 4i..4i+3
// and column 2i+1 in bits 16+4i..19+4i, so (word >> 4i) & 0x000F000F is the bf16 pair of
// neighbouring columns that the tensor cores take, up to the exponent.
#pragma once

#include "common.cuh"

namespace moe {

struct W4Matrix {
  const uint8_t* codes;         // [n, R, K / 2]
  const __nv_bfloat16* scales;  // [n, ceil(K / G), R]
};

// One class of products  out rows = epi(rows . W_g^T): group g multiplies its rows with
// matrix g.
struct W4Class {
  int n_groups;
  int R;                 // weight rows (output features) of a matrix
  int K;                 // reduction length, a multiple of 32
  const int* seg_off;    // device [n_groups + 1]: rows of group g (nullable)
  int max_row;           // seg_off entries and perm values lie in [0, max_row]
  int const_rows;        // rows per group when seg_off == nullptr
  int b_group_stride;    // first input row of group g, and its first output row, when
  int out_group_stride;  //   seg_off == nullptr
  const __nv_bfloat16* b;  // input rows [b_rows, K]
  long long b_rows;
  W4Matrix a0, a1;       // a1: the up matrix (SwiGLU)
  void* out;             // bf16 rows (SWIGLU, RELU) or fp32 rows (DOWN), pitch R
  const float* row_w;    // DOWN: weight of an output row (nullable; preferred over task_w)
  const float* task_w;   // DOWN: weight task_w[perm[row]] (nullable: 1)
  const int* perm;
};

constexpr int W4_MAX_CTAS = 160;              // CTAs of a launch
constexpr int W4_COUNTERS = W4_MAX_CTAS * 8;  // one an epilogue warp: a product's cut tiles
constexpr int W4_COUNTERS2 = W4_MAX_CTAS * 4; // the same where one launch does both products
constexpr unsigned long long W4_COUNT = 1024; // what a launch of both products counts: more than its epilogue warps
// Counter words of a workspace: two sets that the launches of the two products use in
// turn; for launches that do both, four of each kind of grid (even and odd launches, first
// and second product), as each kind counts its own launches.
constexpr int W4_GRID_KINDS = 2;
constexpr int W4_COUNTER_WORDS = 2 * W4_COUNTERS + W4_GRID_KINDS * 4 * W4_COUNTERS2;

struct W4Params {
  W4Class cls[4];  // [product][routed, shared]; launches of one product use the first two
  int n_classes;
  int group;    // 32, 64 or 128
  float* partial;           // w4_partial_bytes(): sums of tiles that CTAs share
  // warps that have left their sums of a tile, zero before the launch
  unsigned* counters;       // [W4_COUNTERS], or the four sets of W4_COUNTERS2 of this kind
  // [W4_COUNTERS]: zeroed here, used by the next product (a tile's last warp zeroes its own
  // counter; this is for what a launch leaves whose waits ran out)
  unsigned* counters_next;
  unsigned long long* grid_count;  // both products: epilogue warps that have left the first
  int* status;
  unsigned long long wait_limit_ns;
  unsigned stall;  // test hook, 0 but for tests of the time limits (moe_debug_set_barrier_extra)
};

// Input rows of a tile (16 .. 192; 192 stands for 224 where w4_deep says so) for segments of
// at most T and on average avg_rows rows.
int w4_pick_bn(long long T, double avg_rows);
constexpr size_t w4_partial_floats(int bn) { return (size_t)W4_MAX_CTAS * 2 * bn * 128; }  // of one product
size_t w4_partial_bytes(int bn);
// Whether tiles of bn rows take both products in one launch (epi: the first one's, cls all
// four); otherwise a launch each.
bool w4_both_products(int bn);
int w4_grid_kind(int bn);  // and of which kind its grid is: one size on a device
cudaError_t launch_w4_gemm(int epi, int bn, const W4Params& p, cudaStream_t s);
cudaError_t launch_quantize_w4(long long n, int rows, int cols, int group, const void* src, uint8_t* codes,
                               void* scales, cudaStream_t s);
cudaError_t launch_dequantize_w4(long long n, int rows, int cols, int group, const uint8_t* codes, const void* scales,
                                 void* dst, cudaStream_t s);

}  // namespace moe
