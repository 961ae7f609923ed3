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
struct Vec8;  // 8 consecutive elements

template <>
struct Vec8<__nv_bfloat16> {
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
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(void* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Reduction over the TPR threads of a row; TPR > 32 goes through shared memory (`buf`,
// one slot a warp; the caller passes a buffer of its own to each reduction, so one
// barrier each is enough).
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* buf) {
#pragma unroll
  for (int off = (TPR < 32 ? TPR : 32) / 2; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = MAX ? fmaxf(v, buf[i]) : v + buf[i];
  }
  return v;
}

// TPR threads a row (32: several rows a block, one a warp; more: one row a block), VPT
// vectors of 8 elements a thread, vector i of thread t at 8 (i TPR + t). An element is
// read and written by the same thread, in that order, so sum_out or y may be x or
// residual themselves.
template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
    add_rmsnorm_kernel(long long rows, int d, float eps, const T* x, const T* residual,
                       const T* __restrict__ weight, T* sum_out, T* y, uint8_t* __restrict__ codes,
                       float* __restrict__ scales) {
  constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
  __shared__ float red[2][32];
  const int t = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
  const int nv = d >> 3;
  pdl_launch_dependents();
  pdl_wait();
  if (row >= rows) return;  // whole warps (TPR = 32); a block of TPR > 32 has one row
  // the weight row is fetched with the inputs, so its latency is theirs; rows of four
  // vectors a thread fetch it where it is used (registers)
  constexpr bool EARLY = VPT < 4;
  Vec8<T> w[EARLY ? VPT : 1];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (EARLY && i * TPR + t < nv) w[i].load(weight + 8 * (size_t)(i * TPR + t));
  const size_t base = (size_t)row * d;
  float r[VPT][8];
  {
    Vec8<T> a[VPT], b[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * TPR + t < nv) {
        a[i].load(x + base + 8 * (size_t)(i * TPR + t));
        if (residual) b[i].load(residual + base + 8 * (size_t)(i * TPR + t));
      }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (i * TPR + t < nv) {
        a[i].get(r[i]);
        if (residual) {
          float q[8];
          b[i].get(q);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i][j] += q[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = 0.f;
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
  if (sum_out) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * TPR + t < nv) {
        Vec8<T> o;
        o.put(r[i]);
        o.store(sum_out + base + 8 * (size_t)(i * TPR + t));
      }
  }
  ss = row_reduce<TPR, false>(ss, red[0]);
  const float inv = 1.f / sqrtf(ss / (float)d + eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (i * TPR + t < nv) {
      float g[8];
      if (!EARLY) w[0].load(weight + 8 * (size_t)(i * TPR + t));
      w[EARLY ? i : 0].get(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[i][j] = r[i][j] * inv * g[j];
        amax = fmaxf(amax, fabsf(r[i][j]));
      }
      if (y) {
        Vec8<T> o;
        o.put(r[i]);
        o.store(y + base + 8 * (size_t)(i * TPR + t));
      }
    }
  if (codes) {
    amax = row_reduce<TPR, true>(amax, red[1]);
    const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    if (t == 0) scales[row] = sc;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * TPR + t < nv) {
        uint32_t o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          o[h] = 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[h] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(r[i][4 * h + j], sc), __NV_SATFINITE, __NV_E4M3)
                    << (8 * j);
        }
        *reinterpret_cast<uint2*>(codes + base + 8 * (size_t)(i * TPR + t)) = make_uint2(o[0], o[1]);
      }
  }
}

template <typename T, int TPR, int VPT>
cudaError_t launch_norm(long long rows, int d, float eps, const void* x, const void* residual, const void* weight,
                        void* sum_out, void* y, uint8_t* codes, float* scales, cudaStream_t s) {
  constexpr int THREADS = TPR < 128 ? 128 : TPR, RPB = THREADS / TPR;
  const long long blocks = (rows + RPB - 1) / RPB;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = launch_k(add_rmsnorm_kernel<T, TPR, VPT>, dim3((unsigned)blocks), dim3(THREADS), 0, s, rows, d, eps,
                           (const T*)x, (const T*)residual, (const T*)weight, (T*)sum_out, (T*)y, codes, scales);
  count_launch();
  return e;
}

template <typename T>
cudaError_t pick_norm(long long rows, int d, float eps, const void* x, const void* residual, const void* weight,
                      void* sum_out, void* y, uint8_t* codes, float* scales, cudaStream_t s) {
  const int nv = d / 8;
#define MOE_NORM(TPR_, VPT_) \
  if (nv <= TPR_ * VPT_) return launch_norm<T, TPR_, VPT_>(rows, d, eps, x, residual, weight, sum_out, y, codes, scales, s);
  MOE_NORM(32, 1)
  MOE_NORM(32, 2)
  MOE_NORM(128, 1)
  MOE_NORM(128, 2)
  MOE_NORM(256, 2)
  MOE_NORM(512, 2)
  MOE_NORM(1024, 2)
  MOE_NORM(1024, 4)
#undef MOE_NORM
  return cudaErrorInvalidValue;
}

}  // namespace

int norm_max_d() { return 1024 * 4 * 8; }

cudaError_t launch_add_rmsnorm(int dtype, long long rows, int d, float eps, const void* x, const void* residual,
                               const void* weight, void* sum_out, void* y, uint8_t* codes, float* scales,
                               cudaStream_t s) {
  return dtype == MOE_F32
             ? pick_norm<float>(rows, d, eps, x, residual, weight, sum_out, y, codes, scales, s)
             : pick_norm<__nv_bfloat16>(rows, d, eps, x, residual, weight, sum_out, y, codes, scales, s);
}

}  // namespace moe
