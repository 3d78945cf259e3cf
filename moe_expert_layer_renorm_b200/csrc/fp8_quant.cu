// FP8 (E4M3) with one fp32 scale per block of 128: rows of activations in
// groups of 128 along K, weights in blocks of 128 x 128.
//   m = max(max |x_i| over the block, 2^-100)     (a NaN is left out)
//   s = m / 448
//   q_i = e4m3_rne_sat((448 x_i) / m)             value q_i s
// The product 448 x_i comes first and is then divided by m (quotient_by): for
// bf16 and f16 inputs 448 x_i is exact in fp32, so a
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

static inline int fp8_blocks(int n) { return int((unsigned(n) + kFp8Block - 1) / kFp8Block); }

// The block's factors: code = e4m3((x * mul) / div).
struct Fp8Scale {
  float mul, div, scale, rcp;   // mul: 448, or 448 2^-32; rcp: 1 / div, rounded to nearest
};
// n / d to nearest, given rcp = 1 / d rounded to nearest: the product with it is
// within two steps of the quotient, its remainder is exact in one fma, and
// the second fma adds the remainder's share (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  What
// matters here is that a quotient that fp32 holds comes out exactly.
__device__ __forceinline__ float quotient_by(float n, float d, float rcp) {
  const float q = __fmul_rn(n, rcp);
  return __fmaf_rn(__fmaf_rn(-q, d, n), rcp, q);
}
__device__ __forceinline__ Fp8Scale fp8_scale_of(float amax) {
  Fp8Scale f;
  const float m = fmaxf(amax, kFp8Floor);
  const bool big = m >= 0x1p100f, inf = m > 3.4028235e38f;
  f.mul = big ? kFp8Max * 0x1p-32f : kFp8Max;
  f.div = big ? m * 0x1p-32f : m;
  f.scale = inf ? m : quotient_by(m, kFp8Max, 1.0f / kFp8Max);
  f.rcp = __frcp_rn(f.div);
  // an infinite m: rcp is 0, and with a finite divisor the remainder's share is
  // 0 too, so finite elements become 0 and the infinite ones NaN
  if (inf) f.div = 1.0f;
  return f;
}
// Two values -> two E4M3 codes, the first in the low byte (nearest even,
// saturating at 448; NaN -> 0x7F).
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Pairs of fp32 values in one 64-bit register: the packed operations take one
// issue slot for two results.
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// quotient_by for two values at once.
__device__ __forceinline__ uint32_t fp8_codes2(float a, float b, const Fp8Scale& f) {
  const unsigned long long rcp = pack2(f.rcp, f.rcp), nd = pack2(-f.div, -f.div);
  const unsigned long long t = mul2(pack2(a, b), pack2(f.mul, f.mul)), q = mul2(t, rcp);
  const float2 r = unpack2(fma2(fma2(q, nd, t), rcp, q));
  return cvt_e4m3x2(r.x, r.y);
}
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, const Fp8Scale& f) {
  return fp8_codes2(a, b, f) | (fp8_codes2(c, d, f) << 16);
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

// Sixteen consecutive values, as loaded.  The vector loads stand in one
// straight run, before the first conversion: behind a branch each, with their
// conversions, they would wait for one another.
template <typename T>
struct Raw16 {
  static constexpr int kWords = sizeof(T) * 16 / 16;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* p) {   // 16-byte aligned, all present
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void load_some(const T* p, int n) {   // the first n of them, zeros after
    T* e = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < 16; ++i) e[i] = i < n ? p[i] : T(0.0f);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void to(float (&v)[16]) const {
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = to_f32<T>(e[i]);
  }
};

// One group of 128 values, held by eight lanes, 16 each.
__device__ __forceinline__ float group_max(const float (&v)[16]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));   // fmaxf leaves NaN out
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  return m;
}
__device__ __forceinline__ uint4 fp8_codes16(const float (&v)[16], const Fp8Scale& f) {
  return make_uint4(fp8_codes4(v[0], v[1], v[2], v[3], f), fp8_codes4(v[4], v[5], v[6], v[7], f),
                    fp8_codes4(v[8], v[9], v[10], v[11], f), fp8_codes4(v[12], v[13], v[14], v[15], f));
}

// Rows: eight lanes take one group at a time, the grid striding over all
// groups with the next group's loads in flight behind one group's arithmetic.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const T* __restrict__ x, int M, int K, long long ld_x,
                                                             uint8_t* __restrict__ codes, long long ld_codes,
                                                             float* __restrict__ scales, long long ld_scales) {
  pdl_enter();
  const uint32_t nb = (uint32_t(K) + kFp8Block - 1) / kFp8Block, groups = uint32_t(M) * nb;   // < 2^31
  const uint32_t stride = gridDim.x * 32u;
  const int sub = threadIdx.x & 7;
  Raw16<T> raw;
  uint32_t row = 0, b = 0;
  auto fetch = [&](uint32_t g) {   // the whole warp: eight-lane sets past the end read nothing
    row = g / nb;
    b = g - row * nb;
    const int k0 = b * kFp8Block + sub * 16;
    const T* src = x + row * ld_x + k0;
    if (__all_sync(0xFFFFFFFFu, VEC && g < groups && (b + 1) * kFp8Block <= K)) {
      raw.load(src);
    } else {
      const int n = g < groups ? K - k0 : 0;
      if (VEC && n >= 16) raw.load(src);
      else raw.load_some(src, n);
    }
  };
  uint32_t g = (blockIdx.x * 256u + threadIdx.x) >> 3;
  const uint32_t warp_first = (blockIdx.x * 256u + (threadIdx.x & ~31u)) >> 3;   // the warp's first group
  fetch(g);
  for (uint32_t w = warp_first; w < groups; w += stride) {
    float v[16];
    raw.to(v);
    const uint32_t r = row, c = b;
    const bool live = g < groups;
    g += stride;
    if (w + stride < groups) fetch(g);
    const Fp8Scale f = fp8_scale_of(group_max(v));
    if (!live) continue;
    if (sub == 0) scales[r * ld_scales + c] = f.scale;
    const int k0 = c * kFp8Block + sub * 16, n = K - k0;
    if (n <= 0) continue;
    const uint4 q = fp8_codes16(v, f);
    uint8_t* dst = codes + r * ld_codes + k0;
    if (n >= 16) {   // ld_codes and codes are multiples of 16
      *reinterpret_cast<uint4*>(dst) = q;
    } else {
      const uint32_t word[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (e < n) dst[e] = uint8_t(word[e >> 2] >> (8 * (e & 3)));
    }
  }
}

// CTAs for that many groups of 128, 32 a CTA and round.
constexpr int kQuantCtas = 12;   // a SM
static unsigned fp8_quant_grid(long long groups, int num_sms) {
  return unsigned(std::min<long long>((groups + 31) / 32, (long long)num_sms * kQuantCtas));
}

template <typename T>
static cudaError_t launch_fp8_quant_t(const void* x, int M, int K, long long ld_x, uint8_t* codes, long long ld_codes,
                                      float* scales, long long ld_scales, cudaStream_t s) {
  const long long groups = (long long)M * fp8_blocks(K);
  const dim3 grid(fp8_quant_grid(groups, device_sm_count()));
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
  const int left = K - k0;   // values of the row from k0 on; k0 plus a place may pass 2^31
  const float* src = w + (long long)n * K + k0;
  float v[64];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    v[i] = n < N && i < left ? __ldg(src + i) : 0.0f;
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
  if (blockIdx.x == 0)
    for (long long c = gridDim.x + threadIdx.x; c < ld_scales; c += blockDim.x)
      scales[(long long)blockIdx.y * ld_scales + c] = 0.0f;
  if (n >= N) return;
  uint8_t* dst = codes + (long long)n * ld_codes + k0;
#pragma unroll
  for (int i = 0; i < 64; i += 4) {
    const uint32_t c = fp8_codes4(v[i], v[i + 1], v[i + 2], v[i + 3], f);
    if (left - i >= 4) {   // codes and ld_codes are multiples of 16
      *reinterpret_cast<uint32_t*>(dst + i) = c;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < left) dst[i + j] = uint8_t(c >> (8 * j));
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
