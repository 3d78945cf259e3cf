// The router's balance loss and per-expert counts, and the gradient of the
// router's logits.  Over the Tv valid tokens, p = softmax(logits[t]):
//   c_e  = number of (t, j) with topk_ids[t, j] = e
//   loss = coef * E / (Tv k) * sum_e c_e * (1 / Tv) sum_t p[t, e]
//   dlogits[t, e] = dloss * coef * E / (Tv^2 k) * p[t, e] (c_e - sum_i p[t, i] c_i)
// and, for the weights w = softmax over a token's k selected logits with the
// gradient dw, dlogits[t, id_j] += w_j (dw_j - sum_i w_i dw_i).
//
// One warp per token, the token's logits in registers: lane l holds the V
// consecutive logits from V (l + 32 i) (V = 4 as one 16-byte load where E, the
// row pitch and the addresses allow it, else 1).
#include <type_traits>

#include "sm100.cuh"

namespace ftmoe {

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}

// softmax of one row into v (places past E hold 0).  A row whose logits are
// all -inf has no probabilities: zeros.
template <int V, int NV>
__device__ __forceinline__ void load_softmax(const float* __restrict__ row, int E, int lane, float (&v)[NV * V]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = V * (lane + 32 * i);
    if constexpr (V == 4) {
      const float4 f = e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    } else {
      v[i] = e < E ? __ldg(row + e) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NV * V; ++i) m = fmaxf(m, v[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;      // all -inf: exp gives zeros
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < NV * V; ++i) {
    v[i] = expf(v[i] - m);
    z += v[i];
  }
  z = warp_sum(z);
  const float inv = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
  for (int i = 0; i < NV * V; ++i) v[i] *= inv;
}

// Partial sums of a CTA's tokens: part_p [grid][E], part_c [grid][E], part_n [grid].
template <int V, int NV>
__global__ void __launch_bounds__(kBalThreads)
balance_partial_kernel(const float* __restrict__ logits, long long ld, const int32_t* __restrict__ ids,
                       const uint8_t* __restrict__ valid, int T, int E, int k, float* __restrict__ part_p,
                       int32_t* __restrict__ part_c, int32_t* __restrict__ part_n) {
  pdl_enter();
  extern __shared__ float bal_smem[];
  float* sums = bal_smem;                                          // [kBalWarps][E]
  int* cnt = reinterpret_cast<int*>(bal_smem + kBalWarps * E);     // [E], then the valid tokens
  for (int e = threadIdx.x; e <= E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[NV * V] = {};
  int n = 0;
  for (int t = blockIdx.x * kBalWarps + warp; t < T; t += gridDim.x * kBalWarps) {
    if (valid && !__ldg(valid + t)) continue;
    ++n;
    if (lane < k) {
      const int e = __ldg(ids + size_t(t) * k + lane);
      if (e >= 0 && e < E) atomicAdd(cnt + e, 1);
      else set_device_status(FT_DEV_BAD_INDEX);
    }
    float p[NV * V];
    load_softmax<V, NV>(logits + t * ld, E, lane, p);
#pragma unroll
    for (int i = 0; i < NV * V; ++i) acc[i] += p[i];
  }
  if (lane == 0) atomicAdd(cnt + E, n);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int e = V * (lane + 32 * i) + c;
      if (e < E) sums[warp * E + e] = acc[i * V + c];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kBalWarps; ++w) s += sums[w * E + e];
    part_p[size_t(blockIdx.x) * E + e] = s;
    part_c[size_t(blockIdx.x) * E + e] = cnt[e];
  }
  if (threadIdx.x == 0) part_n[blockIdx.x] = cnt[E];
}

// Adds the partials in block order and forms the loss (one CTA).
__global__ void __launch_bounds__(1024)
balance_finish_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                      const int32_t* __restrict__ part_n, int blocks, int E, int k, float coef,
                      int32_t* __restrict__ counts, int32_t* __restrict__ n_valid, float* __restrict__ loss) {
  pdl_enter();
  __shared__ float warp_sums[32];
  int n = 0;
  for (int b = 0; b < blocks; ++b) n += part_n[b];
  const int e = threadIdx.x;
  float term = 0.0f;
  if (e < E) {
    float p = 0.0f;
    int c = 0;
    for (int b = 0; b < blocks; ++b) {
      p += part_p[size_t(b) * E + e];
      c += part_c[size_t(b) * E + e];
    }
    counts[e] = c;
    term = float(c) * p;
  }
  term = warp_sum(term);
  if ((e & 31) == 0) warp_sums[e >> 5] = term;
  __syncthreads();
  if (e < 32) {
    const float sum = warp_sum(warp_sums[e]);
    if (e == 0) {
      *n_valid = n;
      *loss = n > 0 ? coef * float(E) / (float(n) * float(n) * float(k)) * sum : 0.0f;
    }
  }
}

// One warp per token; the row's gradient passes through shared memory, where
// the selected experts' own terms are added (in the order j = 0 .. k-1, each
// place by the lane that owns it: repeated ids add up in a fixed order).
template <int V, int NV>
__global__ void __launch_bounds__(kBalThreads)
route_backward_kernel(const float* __restrict__ logits, long long ld, const int32_t* __restrict__ ids,
                      const float* __restrict__ w, const float* __restrict__ dw, const uint8_t* __restrict__ valid,
                      int T, int E, int k, float coef, const int32_t* __restrict__ counts,
                      const int32_t* __restrict__ n_valid, const float* __restrict__ dloss, float* __restrict__ dlogits,
                      long long ldd) {
  pdl_enter();
  extern __shared__ float bal_smem[];
  float* cf = bal_smem;                                  // [E] counts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* srow = bal_smem + E + warp * E;
  float scale = 0.0f;
  if (counts) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) cf[e] = float(counts[e]);
    const float n = float(*n_valid);
    if (n > 0.0f) scale = (dloss ? *dloss : 1.0f) * coef * float(E) / (n * n * float(k));
  }
  __syncthreads();
  for (int t = blockIdx.x * kBalWarps + warp; t < T; t += gridDim.x * kBalWarps) {
    float g[NV * V] = {};
    const bool live = !valid || __ldg(valid + t);
    if (live && counts) {
      load_softmax<V, NV>(logits + t * ld, E, lane, g);
      float mean = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const int e = V * (lane + 32 * i) + c;
          if (e < E) mean = fmaf(g[i * V + c], cf[e], mean);
        }
      mean = warp_sum(mean);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const int e = V * (lane + 32 * i) + c;
          if (e < E) g[i * V + c] *= scale * (cf[e] - mean);
        }
    }
    if (live && dw) {
      const float wj = lane < k ? __ldg(w + size_t(t) * k + lane) : 0.0f;
      const float dj = lane < k ? __ldg(dw + size_t(t) * k + lane) : 0.0f;
      const int id = lane < k ? __ldg(ids + size_t(t) * k + lane) : 0;
      const float mine = wj * (dj - warp_sum(wj * dj));
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const int e = V * (lane + 32 * i) + c;
          if (e < E) srow[e] = g[i * V + c];
        }
      for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(0xFFFFFFFFu, id, j);
        const float add = __shfl_sync(0xFFFFFFFFu, mine, j);
        if (e < 0 || e >= E) {
          if (lane == 0) set_device_status(FT_DEV_BAD_INDEX);
        } else if (((e / V) & 31) == lane) {
          srow[e] += add;
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const int e = V * (lane + 32 * i) + c;
          if (e < E) g[i * V + c] = srow[e];
        }
    }
    float* out = dlogits + t * ldd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = V * (lane + 32 * i);
      if (e >= E) continue;
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(out + e) = make_float4(g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]);
      else
        out[e] = g[i];
    }
  }
}

// ---------------------------------------------------------------- host ---

// Calls f(V, NV) as integral constants for E experts: NV vectors of V logits a lane.
template <typename F>
static cudaError_t balance_variant(int E, bool vec, F f) {
  using std::integral_constant;
  const int nv = (E + 31) / 32;      // logits a lane
  if (vec) {
    if (nv <= 4) return f(integral_constant<int, 4>(), integral_constant<int, 1>());
    if (nv <= 8) return f(integral_constant<int, 4>(), integral_constant<int, 2>());
    if (nv <= 16) return f(integral_constant<int, 4>(), integral_constant<int, 4>());
    return f(integral_constant<int, 4>(), integral_constant<int, 8>());
  }
  if (nv <= 2) return f(integral_constant<int, 1>(), integral_constant<int, 2>());
  if (nv <= 8) return f(integral_constant<int, 1>(), integral_constant<int, 8>());
  return f(integral_constant<int, 1>(), integral_constant<int, 32>());
}

static int balance_blocks(int T, int num_sms) {
  return int(std::min<long long>((T + kBalWarps - 1) / kBalWarps, num_sms));
}
static size_t balance_ws_bytes(int T, int E, int num_sms) {
  return size_t(balance_blocks(T, num_sms)) * (2 * size_t(E) + 1) * 4;
}

static cudaError_t launch_balance(const float* logits, long long ld, const int32_t* ids, const uint8_t* valid, int T,
                                  int E, int k, float coef, int32_t* counts, int32_t* n_valid, float* loss, void* ws,
                                  int num_sms, cudaStream_t s) {
  const int blocks = balance_blocks(T, num_sms);
  float* part_p = static_cast<float*>(ws);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + size_t(blocks) * E);
  int32_t* part_n = part_c + size_t(blocks) * E;
  if (T > 0) {
    const bool vec = E % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
    const cudaError_t e = balance_variant(E, vec, [&](auto v, auto nv) {
      ProfileScope prof(FT_KERNEL_BALANCE, s);
      return launch_pdl(balance_partial_kernel<decltype(v)::value, decltype(nv)::value>, dim3(blocks),
                        dim3(kBalThreads), ((kBalWarps + 1) * size_t(E) + 1) * 4, s, logits, ld, ids, valid, T, E, k,
                        part_p, part_c, part_n);
    });
    if (e != cudaSuccess) return e;
  }
  ProfileScope prof(FT_KERNEL_BALANCE, s);
  return launch_pdl(balance_finish_kernel, dim3(1), dim3(1024), 0, s, static_cast<const float*>(part_p),
                    static_cast<const int32_t*>(part_c), static_cast<const int32_t*>(part_n), blocks, E, k, coef, counts,
                    n_valid, loss);
}

static cudaError_t launch_route_backward(const float* logits, long long ld, const int32_t* ids, const float* w,
                                         const float* dw, const uint8_t* valid, int T, int E, int k, float coef,
                                         const int32_t* counts, const int32_t* n_valid, const float* dloss,
                                         float* dlogits, long long ldd, int num_sms, cudaStream_t s) {
  const bool vec = E % 4 == 0 && ld % 4 == 0 && ldd % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(dlogits) & 15) == 0;
  const int blocks = int(std::min<long long>((T + kBalWarps - 1) / kBalWarps, 4LL * num_sms));
  return balance_variant(E, vec, [&](auto v, auto nv) {
    ProfileScope prof(FT_KERNEL_ROUTE_BACKWARD, s);
    return launch_pdl(route_backward_kernel<decltype(v)::value, decltype(nv)::value>, dim3(blocks), dim3(kBalThreads),
                      (kBalWarps + 1) * size_t(E) * 4, s, logits, ld, ids, w, dw, valid, T, E, k, coef, counts, n_valid,
                      dloss, dlogits, ldd);
  });
}

}  // namespace ftmoe
