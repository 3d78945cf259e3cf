// FP8 (E4M3) with one fp32 scale per block of 128: rows of activations in
// groups of 128 along K, weights in blocks of 128 x 128.
//   m = max(max |x_i| over the block, 2^-100)     (a NaN is left out)
//   s = m / 448
//   q_i = e4m3_rne_sat((448 x_i) / m)             value q_i s
// The product 448 x_i comes first and is then divided by m, one correctly
// rounded division: for bf16 and f16 inputs 448 x_i is exact in fp32, so a
// quotient that lies exactly between two codes is seen as the tie it is and
// goes to the even code (x_i * (448 / m) would round the factor first and
// push every such tie to one side or the other).  A block whose m is above
// 2^100 is brought down by 2^-32 before the product, which is exact for every
// element that does not end as code 0.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sm100.cuh"

namespace ftmoe {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;
constexpr float kFp8Floor = 0x1p-100f;

static inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

// The block's factors: code = e4m3((x * pre * 448) / div).
struct Fp8Scale {
  float pre, div, scale;
};
__device__ __forceinline__ Fp8Scale fp8_scale_of(float amax) {
  Fp8Scale f;
  const float m = fmaxf(amax, kFp8Floor);
  f.pre = m >= 0x1p100f ? 0x1p-32f : 1.0f;
  f.div = m * f.pre;
  f.scale = __fdiv_rn(m, kFp8Max);
  return f;
}
__device__ __forceinline__ float fp8_quotient(float x, const Fp8Scale& f) {
  return __fdiv_rn(__fmul_rn(x * f.pre, kFp8Max), f.div);
}
// The same for values that fp32 arithmetic has just computed (h), by one
// product with 448 / m: no tie of theirs is meant, and a quotient within
// 2^-23 of one may go either way.
__device__ __forceinline__ float fp8_factor_of(const Fp8Scale& f) { return __fdiv_rn(kFp8Max, f.div) * f.pre; }
// Two values -> two E4M3 codes, the first in the low byte (nearest even,
// saturating at 448; NaN -> 0x7F).
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, const Fp8Scale& f) {
  return cvt_e4m3x2(fp8_quotient(a, f), fp8_quotient(b, f)) |
         (cvt_e4m3x2(fp8_quotient(c, f), fp8_quotient(d, f)) << 16);
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

// Eight consecutive values at p (VEC: 16-byte aligned and all present), else
// the first n of them, zeros after.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
  if (VEC && n >= 8) {
    constexpr int kWords = sizeof(T) * 8 / 16;
    uint4 w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32<T>(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ float absmax8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));   // fmaxf leaves NaN out
  return m;
}

// Rows: sixteen lanes take one group of 128 values, eight each.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const T* __restrict__ x, int M, int K, long long ld_x,
                                                             uint8_t* __restrict__ codes, long long ld_codes,
                                                             float* __restrict__ scales, long long ld_scales) {
  pdl_enter();
  const int nb = (K + kFp8Block - 1) / kFp8Block;
  const long long g = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 4;
  const bool live = g < (long long)M * nb;
  const int sub = threadIdx.x & 15;
  const long long row = live ? g / nb : 0;
  const int b = live ? int(g - row * nb) : 0;
  const int k0 = b * kFp8Block + sub * 8;
  const int n = live ? min(8, K - k0) : 0;
  float v[8];
  load8<T, VEC>(x + row * ld_x + k0, n, v);
  float m = absmax8(v);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  if (!live) return;
  const Fp8Scale f = fp8_scale_of(m);
  if (sub == 0) scales[row * ld_scales + b] = f.scale;
  if (n <= 0) return;
  const uint32_t c0 = fp8_codes4(v[0], v[1], v[2], v[3], f), c1 = fp8_codes4(v[4], v[5], v[6], v[7], f);
  uint8_t* dst = codes + row * ld_codes + k0;
  if (n == 8) {   // ld_codes and codes are multiples of 16: dst is 8-byte aligned
    *reinterpret_cast<uint2*>(dst) = make_uint2(c0, c1);
  } else {
    for (int i = 0; i < n; ++i) dst[i] = uint8_t((i < 4 ? c0 : c1) >> (8 * (i & 3)));
  }
}

template <typename T>
static cudaError_t launch_fp8_quant_t(const void* x, int M, int K, long long ld_x, uint8_t* codes, long long ld_codes,
                                      float* scales, long long ld_scales, cudaStream_t s) {
  const long long threads = 16LL * M * fp8_blocks(K);
  const dim3 grid(unsigned((threads + 255) / 256));
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (ld_x * sizeof(T)) % 16 == 0;
  ProfileScope prof(FT_KERNEL_FP8_QUANT, s);
  return launch_pdl(vec ? fp8_quant_rows_kernel<T, true> : fp8_quant_rows_kernel<T, false>, grid, dim3(256), 0, s,
                    static_cast<const T*>(x), M, K, ld_x, codes, ld_codes, scales, ld_scales);
}
static cudaError_t launch_fp8_quant(const void* x, int x_type, int M, int K, long long ld_x, uint8_t* codes,
                                    long long ld_codes, float* scales, long long ld_scales, cudaStream_t s) {
  auto f = x_type == FT_F32 ? launch_fp8_quant_t<float>
         : x_type == FT_BF16 ? launch_fp8_quant_t<__nv_bfloat16> : launch_fp8_quant_t<__half>;
  return f(x, M, K, ld_x, codes, ld_codes, scales, ld_scales, s);
}

// Weights: one CTA per 128 x 128 block, 64 values a thread (threads 2r and
// 2r + 1 share row r), held in registers between the maximum and the codes.
// Padding columns of the scale rows are zeroed.
__global__ void __launch_bounds__(256) fp8_pack_kernel(const float* __restrict__ w, int N, int K,
                                                       uint8_t* __restrict__ codes, long long ld_codes,
                                                       float* __restrict__ scales, int ld_scales) {
  pdl_enter();
  __shared__ float warp_max[8];
  const int n = blockIdx.y * kFp8Block + (threadIdx.x >> 1);
  const int k0 = blockIdx.x * kFp8Block + (threadIdx.x & 1) * 64;
  const float* src = w + (long long)n * K + k0;
  float v[64];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    v[i] = n < N && k0 + i < K ? __ldg(src + i) : 0.0f;
    m = fmaxf(m, fabsf(v[i]));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, warp_max[i]);
  const Fp8Scale f = fp8_scale_of(m);
  if (threadIdx.x == 0) scales[(long long)blockIdx.y * ld_scales + blockIdx.x] = f.scale;
  if (blockIdx.x == 0 && int(gridDim.x + threadIdx.x) < ld_scales)
    for (int c = gridDim.x + threadIdx.x; c < ld_scales; c += blockDim.x)
      scales[(long long)blockIdx.y * ld_scales + c] = 0.0f;
  if (n >= N) return;
  uint8_t* dst = codes + (long long)n * ld_codes + k0;
#pragma unroll
  for (int i = 0; i < 64; i += 4) {
    const uint32_t c = fp8_codes4(v[i], v[i + 1], v[i + 2], v[i + 3], f);
    if (k0 + i + 4 <= K) {   // codes and ld_codes are multiples of 16
      *reinterpret_cast<uint32_t*>(dst + i) = c;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k0 + i + j < K) dst[i + j] = uint8_t(c >> (8 * j));
    }
  }
}

static cudaError_t launch_fp8_pack(const float* w, int N, int K, uint8_t* codes, long long ld_codes, float* scales,
                                   int ld_scales, cudaStream_t s) {
  ProfileScope prof(FT_KERNEL_PACK, s);
  return launch_pdl(fp8_pack_kernel, dim3(fp8_blocks(K), fp8_blocks(N)), dim3(256), 0, s, w, N, K, codes, ld_codes,
                    scales, ld_scales);
}

}  // namespace ftmoe
