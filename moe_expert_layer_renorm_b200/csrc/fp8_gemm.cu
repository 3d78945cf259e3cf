// Products of E4M3 operands with fp32 block scales:
//   out[r, n] = sum_b sA[r, b] sB[n / 128, b] (sum_{k in block b} qA[r, k] qB[n, k])
// the inner sum and the outer one in fp32.
//
// One thread per output; a warp's lanes take consecutive n of one row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sm100.cuh"

namespace ftmoe {

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// sum over K of one output, K in blocks of 128.
__device__ float fp8_dot(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb, int K) {
  float sum = 0.0f;
  for (int k0 = 0; k0 < K; k0 += kFp8Block) {
    float part = 0.0f;
    const int k1 = min(K, k0 + kFp8Block);
    int k = k0;
    for (; k + 2 <= k1; k += 2) {
      const float2 x = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(a + k));
      const float2 y = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(b + k));
      part = fmaf(x.y, y.y, fmaf(x.x, y.x, part));
    }
    if (k < k1) part = fmaf(e4m3x2_to_f32(a[k]).x, e4m3x2_to_f32(b[k]).x, part);
    sum = fmaf(part, sa[k0 / kFp8Block] * sb[k0 / kFp8Block], sum);
  }
  return sum;
}

__device__ __forceinline__ void store_as(void* out, int type, size_t i, float v) {
  if (type == FT_F32) static_cast<float*>(out)[i] = v;
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

struct Fp8Mat {          // codes and scales of one weight matrix (of slot 0)
  const uint8_t* codes;
  const float* scales;
  long long ld, ld_scales;
};

__global__ void __launch_bounds__(256) fp8_gemm_kernel(const uint8_t* a, long long lda, const float* sa,
                                                       long long ld_sa, const Fp8Mat b, int M, int N, int K,
                                                       void* out, int out_type, long long ldo) {
  pdl_enter();
  const int n = blockIdx.x * 32 + (threadIdx.x & 31);
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (n >= N || r >= M) return;
  const float v = fp8_dot(a + r * lda, sa + r * ld_sa, b.codes + n * b.ld, b.scales + (n / kFp8Block) * b.ld_scales, K);
  store_as(out, out_type, size_t(r) * ldo + n, v);
}

// Rows grouped by expert; up null: out = rows x gate^T, else h = silu(gate) * up (fp32).
__global__ void __launch_bounds__(256)
fp8_grouped_kernel(const uint8_t* a, const float* sa, const int32_t* __restrict__ perm_src, int k_top, int T,
                   const int32_t* __restrict__ offsets, const int32_t* __restrict__ slot_table, int E, int num_slots,
                   long long slot_bytes, const Fp8Mat w0, const Fp8Mat w1, int P, int N, int K, void* out,
                   int out_type) {
  pdl_enter();
  const int n = blockIdx.x * 32 + (threadIdx.x & 31);
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (n >= N || r >= P) return;
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= r) lo = mid; else hi = mid;
  }
  if (r < offsets[lo] || r >= offsets[lo + 1]) return;   // behind the last group
  const int slot = slot_table[lo];
  if (slot < 0) { set_device_status(FT_DEV_NOT_RESIDENT); return; }
  if (slot >= num_slots) { set_device_status(FT_DEV_BAD_INDEX); return; }
  int src = r;
  if (perm_src) {
    src = perm_src[r] / k_top;
    if (src < 0 || src >= T || perm_src[r] < 0) {
      set_device_status(FT_DEV_BAD_INDEX);
      store_as(out, out_type, size_t(r) * N + n, 0.0f);
      return;
    }
  }
  const int kb = (K + kFp8Block - 1) / kFp8Block;
  const uint8_t* x = a + size_t(src) * K;
  const float* sx = sa + size_t(src) * kb;
  auto dot = [&](const Fp8Mat& w) {
    const uint8_t* codes = w.codes + slot * slot_bytes;
    const float* scales = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(w.scales) + slot * slot_bytes);
    return fp8_dot(x, sx, codes + n * w.ld, scales + (n / kFp8Block) * w.ld_scales, K);
  };
  float v = dot(w0);
  if (w1.codes) v = v / (1.0f + __expf(-v)) * dot(w1);
  store_as(out, out_type, size_t(r) * N + n, v);
}

// ---------------------------------------------------------------- host ---

static size_t fp8_gemm_ws_bytes(int, int, int) { return 0; }

static cudaError_t launch_fp8_gemm(const uint8_t* a, long long lda, const float* sa, long long ld_sa, const uint8_t* b,
                                   long long ldb, const float* sb, long long ld_sb, int M, int N, int K, void* out,
                                   int out_type, long long ldo, void*, cudaStream_t s, const char**) {
  ProfileScope prof(FT_KERNEL_FP8_GEMM, s);
  return launch_pdl(fp8_gemm_kernel, dim3((N + 31) / 32, (M + 7) / 8), dim3(256), 0, s, a, lda, sa, ld_sa,
                    Fp8Mat{b, sb, ldb, ld_sb}, M, N, K, out, out_type, ldo);
}

struct Fp8FfnPlan {
  size_t off_x, off_xs, off_hf, off_h, off_hs, total;
};
static Fp8FfnPlan plan_fp8_ffn(int T, int H, int I, int, int k) {
  Fp8FfnPlan p{};
  const size_t P = size_t(T) * k;
  size_t o = 0;
  p.off_x = o;   o = align256(o + size_t(T) * H);
  p.off_xs = o;  o = align256(o + size_t(T) * fp8_blocks(H) * 4);
  p.off_hf = o;  o = align256(o + P * I * 4);
  p.off_h = o;   o = align256(o + P * I);
  p.off_hs = o;  o = align256(o + P * fp8_blocks(I) * 4);
  p.total = o;
  return p;
}

static cudaError_t launch_fp8_ffn(const void* x, int T, int H, int I, int E, int k, const int32_t* perm_src,
                                  const int32_t* offsets, const int32_t* slot_table, const void* pool_v,
                                  const ft_nvfp4_slot_layout& L, void* out, int out_type, void* ws, cudaStream_t s,
                                  const char**) {
  const Fp8FfnPlan pl = plan_fp8_ffn(T, H, I, E, k);
  const uint8_t* pool = static_cast<const uint8_t*>(pool_v);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int P = T * k;
  float* xs = reinterpret_cast<float*>(w + pl.off_xs);
  float* hs = reinterpret_cast<float*>(w + pl.off_hs);
  auto mat = [&](int m) {
    return Fp8Mat{pool + L.codes_off[m], reinterpret_cast<const float*>(pool + L.scales_off[m]), m == FT_DOWN ? I : H,
                  L.ld_scale[m] / 4};
  };
  cudaError_t e = launch_fp8_quant(x, FT_BF16, T, H, H, w + pl.off_x, H, xs, fp8_blocks(H), s);
  if (e != cudaSuccess) return e;
  {
    ProfileScope prof(FT_KERNEL_FP8_GATE_UP, s);
    e = launch_pdl(fp8_grouped_kernel, dim3((I + 31) / 32, (P + 7) / 8), dim3(256), 0, s, w + pl.off_x, xs, perm_src, k,
                   T, offsets, slot_table, E, L.num_slots, (long long)L.slot_bytes, mat(FT_GATE), mat(FT_UP), P, I, H,
                   w + pl.off_hf, int(FT_F32));
  }
  if (e != cudaSuccess) return e;
  e = launch_fp8_quant(w + pl.off_hf, FT_F32, P, I, I, w + pl.off_h, I, hs, fp8_blocks(I), s);
  if (e != cudaSuccess) return e;
  ProfileScope prof(FT_KERNEL_FP8_DOWN, s);
  return launch_pdl(fp8_grouped_kernel, dim3((H + 31) / 32, (P + 7) / 8), dim3(256), 0, s, w + pl.off_h, hs,
                    static_cast<const int32_t*>(nullptr), 1, P, offsets, slot_table, E, L.num_slots,
                    (long long)L.slot_bytes, mat(FT_DOWN), Fp8Mat{}, P, H, I, out, out_type);
}

}  // namespace ftmoe
