// Residual addition, root-mean-square norm and 8-bit output in one pass over the rows
// (the entry of a block that ends in the MoE layer):
//   r = x + residual;  y = r / sqrt(mean(r^2) + eps) * weight;  E4M3 codes of y with
//   scale = max |y| / 448 per row (the format of moe_quantize_e4m3).
// One group of threads holds a whole row in registers (fp32), so every input is read
// once and every output written once: the kernel is bound by HBM for long batches and
// by one load -> two reductions -> store latency for a few rows. Squares, their sum, the
// sum r and y stay in fp32; each output is rounded once (the codes are taken from the
// fp32 y, not from its bf16 rounding).
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

namespace {

template <typename T>
struct Vec;  // the N consecutive elements of 16 bytes

template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  uint4 v;
  __device__ __forceinline__ void load(const void* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Vec<float> {
  static constexpr int N = 4;
  float4 v;
  __device__ __forceinline__ void load(const void* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<float4*>(p) = v; }
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w; }
  __device__ __forceinline__ void put(const float (&f)[4]) { v = make_float4(f[0], f[1], f[2], f[3]); }
};

// Reduction over the threads of a row: one warp, or (WIDE) the block, through shared
// memory (`buf`, one slot a warp; the caller passes a buffer of its own to each
// reduction, so one barrier each is enough).
template <bool WIDE, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* buf) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  if (WIDE) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
    const int nw = blockDim.x >> 5;
    for (int i = 1; i < nw; ++i) v = MAX ? fmaxf(v, buf[i]) : v + buf[i];
  }
  return v;
}

// The code of v / s that an IEEE division gives (moe_quantize_e4m3's: the same row and scale
// have the same codes): with r the rounded reciprocal of s, q = v r is off by less than two
// units in the last place, which at a tie between two codes decides; one step of Markstein's
// method, q + (v - q s) r with the remainder exact in a fused multiply-add, corrects it.
// (The theorem wants a q within one unit; for every mantissa of s, every tie and the numbers
// v around it the corrected quotient was compared with the division's: no other one. A
// division an element took 29.3 us for 4096 x 4096 bf16 rows, v r alone 25.7, this 26.7.)
// Quotients far below E4M3's smallest tie, 2^-10, may be off.
__device__ __forceinline__ float quotient(float v, float s, float r) {
  const float q = v * r;
  return copysignf(fmaf(fmaf(-q, s, v), r, q), v);  // (a quotient of -0 keeps its sign)
}

// A row's threads: a warp (narrow rows, several a block) or (WIDE) the block, of as many
// warps as the row's 16-byte vectors fill, VPT a thread (with a power of two of threads,
// half of them idle at 2056 fp32 elements, 8191 rows took 32 us, so 27).
// Vector i of thread t starts at element N (i TPR + t). An element is read and written by the same thread, in that
// order, so sum_out or y may be x or residual themselves.
// MIN_BLOCKS keeps the registers that the rare rows of large and small squares would take
// from costing the others a block an SM.
template <typename T, bool WIDE, int VPT, int MAX_THREADS,
          int MIN_BLOCKS = !WIDE                             ? (VPT == 1 ? 16 : 10)
                           : VPT == 2                        ? (MAX_THREADS == 256 ? 5 : 3)
                           : VPT == 1 || MAX_THREADS == 512 ? 2
                                                             : 1>
__global__ void __launch_bounds__(MAX_THREADS, MIN_BLOCKS)
    add_rmsnorm_kernel(long long rows, int d, float eps, const T* x, const T* residual,
                       const T* __restrict__ weight, T* sum_out, T* y, uint8_t* __restrict__ codes,
                       float* __restrict__ scales) {
  __shared__ float red[4][32];
  const int TPR = WIDE ? blockDim.x : 32;
  const int t = WIDE ? threadIdx.x : threadIdx.x & 31;
  const long long row = WIDE ? blockIdx.x : (long long)blockIdx.x * (MAX_THREADS / 32) + (threadIdx.x >> 5);
  constexpr int N = Vec<T>::N;
  const int nv = d / N;
  pdl_launch_dependents();
  pdl_wait();
  if (row >= rows) return;  // whole warps; a WIDE block has one row
  // the weight row is fetched with the inputs, so its latency is theirs; rows of four
  // vectors a thread fetch it where it is used (registers)
  constexpr bool EARLY = VPT < 4;
  Vec<T> w[EARLY ? VPT : 1];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (EARLY && i * TPR + t < nv) w[i].load(weight + N * (size_t)(i * TPR + t));
  const size_t base = (size_t)row * d;
  float r[VPT][N];
  {
    Vec<T> a[VPT], b[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * TPR + t < nv) {
        a[i].load(x + base + N * (size_t)(i * TPR + t));
        if (residual) b[i].load(residual + base + N * (size_t)(i * TPR + t));
      }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (i * TPR + t < nv) {
        a[i].get(r[i]);
        if (residual) {
          float q[N];
          b[i].get(q);
#pragma unroll
          for (int j = 0; j < N; ++j) r[i][j] += q[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) r[i][j] = 0.f;
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) ss = fmaf(r[i][j], r[i][j], ss);
  if (sum_out) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * TPR + t < nv) {
        Vec<T> o;
        o.put(r[i]);
        o.store(sum_out + base + N * (size_t)(i * TPR + t));
      }
  }
  ss = row_reduce<WIDE, false>(ss, red[0]);
  float inv = 1.f / sqrtf(ss / (float)d + eps);
  float amax = 0.f;
  // Squares that may have left fp32's range, above or, beside an eps below 2^-60, below
  // (one verdict a row): the row times a power of two that takes its largest element to
  // [1, 2), and another sum. Rows with an infinity keep inv = 0, rows of zeros what eps
  // gives. (What the test costs the other rows: 4096 x 4096 bf16 26.8 -> 27.0 us, 8191 x
  // 2056 fp32 26.8 -> 27.6, 16 x 4096 within 0.05.)
  if (__builtin_expect(!(inv >= 0x1p-63f && inv <= 0x1p30f), 0)) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) top = fmaxf(top, fabsf(r[i][j]));
    top = row_reduce<WIDE, true>(top, red[2]);
    if (top > 0.f && top <= 3.4028235e38f) {
      const int e = ilogbf(top);
      // 2^-e in two factors: it may be no fp32 number itself
      const float f0 = __int_as_float((127 - e / 2) << 23), f1 = __int_as_float((127 - (e - e / 2)) << 23);
      const float eps_e = eps * f0 * f0 * f1 * f1;
      if (eps_e <= 0x1p100f) {  // (else the squares are nothing beside eps, and inv is right)
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j) {
            r[i][j] = r[i][j] * f0 * f1;
            ss = fmaf(r[i][j], r[i][j], ss);
          }
        inv = 1.f / sqrtf(row_reduce<WIDE, false>(ss, red[3]) / (float)d + eps_e);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (i * TPR + t < nv) {
      float g[N];
      if (!EARLY) w[0].load(weight + N * (size_t)(i * TPR + t));
      w[EARLY ? i : 0].get(g);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        r[i][j] = r[i][j] * inv * g[j];
        amax = fmaxf(amax, fabsf(r[i][j]));
      }
      if (y) {
        Vec<T> o;
        o.put(r[i]);
        o.store(y + base + N * (size_t)(i * TPR + t));
      }
    }
  if (codes) {
    amax = row_reduce<WIDE, true>(amax, red[1]);
    float sc = __fdiv_rn(amax, 448.f);
    if (sc == 0.f) sc = 1.f;  // a row of zeros, or one whose scale would be below 2^-150: its codes are zeros
    if (t == 0) scales[row] = sc;
    if (sc < 0x1p-64f) {  // the reciprocal or a remainder of a tiny scale would leave fp32's range
      sc *= 0x1p64f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) r[i][j] *= 0x1p64f;
    }
    const float rs = __frcp_rn(sc);
    if (rs == 0.f) sc = 0.f;  // an infinite scale: finite v give zeros, infinite ones NaN
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * TPR + t < nv) {
        uint32_t o[N / 4];
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
          const float* v = &r[i][4 * h];
          o[h] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(quotient(v[0], sc, rs), quotient(v[1], sc, rs)), __NV_SATFINITE, __NV_E4M3) |
                 (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(quotient(v[2], sc, rs), quotient(v[3], sc, rs)), __NV_SATFINITE, __NV_E4M3)
                     << 16;
        }
        uint8_t* c = codes + base + N * (size_t)(i * TPR + t);
        if constexpr (N == 8)
          *reinterpret_cast<uint2*>(c) = make_uint2(o[0], o[1]);
        else
          *reinterpret_cast<uint32_t*>(c) = o[0];
      }
  }
}

template <typename T, bool WIDE, int VPT, int MAX_THREADS>
cudaError_t launch_norm(int threads, long long rows, int d, float eps, const void* x, const void* residual,
                        const void* weight, void* sum_out, void* y, uint8_t* codes, float* scales, cudaStream_t s) {
  const int per_block = WIDE ? 1 : MAX_THREADS / 32;
  const long long blocks = (rows + per_block - 1) / per_block;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = launch_k(add_rmsnorm_kernel<T, WIDE, VPT, MAX_THREADS>, dim3((unsigned)blocks), dim3(threads), 0, s,
                           rows, d, eps, (const T*)x, (const T*)residual, (const T*)weight, (T*)sum_out, (T*)y, codes,
                           scales);
  count_launch();
  return e;
}

// A warp a row up to two vectors a lane; then two vectors a thread (one where there are
// too few rows to fill the SMs and latency is what counts), four or eight for rows that
// would take more than 512 threads (2048 x 16384 bf16 rows with two of 1024 threads ran at
// 4.3 TB/s, one block a SM).
template <typename T>
cudaError_t pick_norm(long long rows, int d, float eps, const void* x, const void* residual, const void* weight,
                      void* sum_out, void* y, uint8_t* codes, float* scales, cudaStream_t s) {
  const int nv = d / Vec<T>::N;
  const bool few = rows < 2LL * num_sms();
  const int vpt = nv <= 32 ? 1 : nv <= 64 ? 2 : few && nv <= 1024 ? 1 : nv <= 1024 ? 2 : nv <= 4096 ? 4 : 8;
  const int threads = ((nv + vpt - 1) / vpt + 31) & ~31;
#define MOE_NORM(WIDE_, VPT_, MAX_)                                                                              \
  return launch_norm<T, WIDE_, VPT_, MAX_>(WIDE_ ? threads : MAX_, rows, d, eps, x, residual, weight, sum_out, y, \
                                           codes, scales, s)
  if (nv <= 32) MOE_NORM(false, 1, 128);
  if (nv <= 64) MOE_NORM(false, 2, 128);
  if (vpt == 1) MOE_NORM(true, 1, 1024);
  if (vpt == 2) {
    if (threads <= 256) MOE_NORM(true, 2, 256);
    MOE_NORM(true, 2, 512);
  }
  if (vpt == 4) {
    if (threads <= 512) MOE_NORM(true, 4, 512);
    MOE_NORM(true, 4, 1024);
  }
  if constexpr (Vec<T>::N == 4) MOE_NORM(true, 8, 1024);
#undef MOE_NORM
  return cudaErrorInvalidValue;
}

}  // namespace

int norm_max_d() { return 32768; }

cudaError_t launch_add_rmsnorm(int dtype, long long rows, int d, float eps, const void* x, const void* residual,
                               const void* weight, void* sum_out, void* y, uint8_t* codes, float* scales,
                               cudaStream_t s) {
  return dtype == MOE_F32
             ? pick_norm<float>(rows, d, eps, x, residual, weight, sum_out, y, codes, scales, s)
             : pick_norm<__nv_bfloat16>(rows, d, eps, x, residual, weight, sum_out, y, codes, scales, s);
}

}  // namespace moe
