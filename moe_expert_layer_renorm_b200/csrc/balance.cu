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

#include "cluster.cuh"
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

// This lane's logits of one row (places past E hold -inf).
template <int V, int NV>
__device__ __forceinline__ void load_logits(const float* __restrict__ row, int E, int lane, float (&v)[NV * V]) {
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
}
// This lane's places of a row (16-byte pieces for V = 4; 0 past E).
template <int V, int NV>
__device__ __forceinline__ void get_row(const float* row, int E, int lane, float (&v)[NV * V]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = V * (lane + 32 * i);
    if constexpr (V == 4) {
      const float4 f = e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    } else {
      v[i] = e < E ? row[e] : 0.0f;
    }
  }
}
template <int V, int NV>
__device__ __forceinline__ void put_row(float* row, int E, int lane, const float (&v)[NV * V]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = V * (lane + 32 * i);
    if (e >= E) continue;
    if constexpr (V == 4) *reinterpret_cast<float4*>(row + e) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    else row[e] = v[i];
  }
}

// e^(logit - largest logit) in place of the logits (0 past E), and 1 / their
// sum.  A row whose logits are all -inf has no probabilities: zeros and 0.
// expf, as the router: a gradient takes its own p, and the hardware exponential
// would lose 2^-18 of one at e^-80 (8192 x 512, loss and gradient: 22.3 us, with
// it 20.6).
template <int N>
__device__ __forceinline__ void row_exps(float (&v)[N]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;      // all -inf: exp gives zeros
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = expf(v[i] - m);
}
__device__ __forceinline__ float inverse_sum(float z) { return z == 0.0f ? 0.0f : 1.0f / z; }

constexpr int kBalCluster = 8;   // CTAs that add up their sums through distributed shared memory

// Sums over the tokens, in clusters of eight CTAs of W warps: a CTA's warps add up their
// tokens' probabilities in registers, the CTA its warps', and CTA r of a
// cluster the eight CTAs' sums of its eighth of the experts.  All additions
// have a fixed order.  One cluster alone (a small batch) finishes counts and
// loss itself; more of them leave part_p, part_c [clusters][E] and part_n
// [clusters] to balance_finish_kernel.  A token's logits are requested behind
// the token before it.
template <int V, int NV, int W>
__global__ void __cluster_dims__(kBalCluster, 1, 1) __launch_bounds__(32 * W)
balance_kernel(const float* __restrict__ logits, long long ld, const int32_t* __restrict__ ids,
               const uint8_t* __restrict__ valid, int T, int E, int k, float coef, float* __restrict__ part_p,
               int32_t* __restrict__ part_c, int32_t* __restrict__ part_n, int32_t* __restrict__ counts,
               int32_t* __restrict__ n_valid, float* __restrict__ loss) {
  pdl_enter();
  extern __shared__ float bal_smem[];
  float* sums = bal_smem;                                          // [W][E], then [0] the CTA's
  int* cnt = reinterpret_cast<int*>(bal_smem + W * E);     // [E], then the valid tokens
  float* terms = reinterpret_cast<float*>(cnt + E + 1);            // [W]
  float* cta_term = terms + W;                             // [1]
  for (int e = threadIdx.x; e <= E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int step = gridDim.x * W;
  float acc[NV * V] = {};
  int n = 0;
  int t = blockIdx.x * W + warp;
  float next[NV * V];
  bool live = t < T && (!valid || __ldg(valid + t));
  if (live) load_logits<V, NV>(logits + t * ld, E, lane, next);
  for (; t < T; t += step) {
    const bool now = live;
    float p[NV * V];
#pragma unroll
    for (int i = 0; i < NV * V; ++i) p[i] = next[i];
    const int id = now && lane < k ? __ldg(ids + size_t(t) * k + lane) : 0;
    live = t + step < T && (!valid || __ldg(valid + t + step));
    if (live) load_logits<V, NV>(logits + (t + step) * ld, E, lane, next);
    if (!now) continue;
    ++n;
    row_exps(p);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < NV * V; ++i) z += p[i];
    const float inv = inverse_sum(warp_sum(z));
#pragma unroll
    for (int i = 0; i < NV * V; ++i) acc[i] = fmaf(p[i], inv, acc[i]);
    if (lane < k) {
      if (id >= 0 && id < E) atomicAdd(cnt + id, 1);
      else set_device_status(FT_DEV_BAD_INDEX);
    }
  }
  if (lane == 0) atomicAdd(cnt + E, n);
  put_row<V, NV>(sums + warp * E, E, lane, acc);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += sums[w * E + e];
    sums[e] = s;
  }
  cluster_sync();
  const int rank = cluster_rank(), cid = blockIdx.x / kBalCluster;
  const bool one = gridDim.x == kBalCluster;
  const int eighth = (E + kBalCluster - 1) / kBalCluster, e0 = rank * eighth, e1 = min(E, e0 + eighth);
  float term = 0.0f;
  for (int e = e0 + threadIdx.x; e < e1; e += blockDim.x) {
    float ps[kBalCluster];
    int cs[kBalCluster];
#pragma unroll
    for (int r = 0; r < kBalCluster; ++r) {
      ps[r] = ld_cluster_f32(cluster_addr(sums + e, r));
      cs[r] = ld_cluster_s32(cluster_addr(cnt + e, r));
    }
    float p = 0.0f;
    int c = 0;
#pragma unroll
    for (int r = 0; r < kBalCluster; ++r) { p += ps[r]; c += cs[r]; }
    if (one) {
      counts[e] = c;
      term += float(c) * p;
    } else {
      part_p[size_t(cid) * E + e] = p;
      part_c[size_t(cid) * E + e] = c;
    }
  }
  int total = 0;
  if (rank == 0 && threadIdx.x == 0)
    for (int r = 0; r < kBalCluster; ++r) total += ld_cluster_s32(cluster_addr(cnt + E, r));
  if (!one) {
    if (rank == 0 && threadIdx.x == 0) part_n[cid] = total;
    cluster_sync();   // no CTA leaves while another reads its sums
    return;
  }
  term = warp_sum(term);
  if (lane == 0) terms[warp] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int w = 0; w < W; ++w) s += terms[w];
    *cta_term = s;
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float s = 0.0f;
    for (int r = 0; r < kBalCluster; ++r) s += ld_cluster_f32(cluster_addr(cta_term, r));
    *n_valid = total;
    *loss = total > 0 ? coef * float(E) / (float(total) * float(total) * float(k)) * s : 0.0f;
  }
  cluster_sync();
}

// Adds the clusters' sums in their order and forms the loss (one CTA of 1024
// threads: as many threads an expert as fit, each an even share of the clusters).
__global__ void __launch_bounds__(1024)
balance_finish_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                      const int32_t* __restrict__ part_n, int clusters, int E, int k, float coef,
                      int32_t* __restrict__ counts, int32_t* __restrict__ n_valid, float* __restrict__ loss) {
  pdl_enter();
  __shared__ float sp[1024], warp_sums[32];
  __shared__ int sc[1024];
  const int slices = 1024 / E, slice = threadIdx.x / E, e = threadIdx.x - slice * E;
  const int share = (clusters + slices - 1) / slices, c0 = slice * share, c1 = min(clusters, c0 + share);
  int n = 0;
  if (threadIdx.x < 32) {
    for (int b = threadIdx.x; b < clusters; b += 32) n += part_n[b];
    n = __reduce_add_sync(0xFFFFFFFFu, n);
  }
  if (slice < slices) {
    float p = 0.0f;
    int c = 0;
    for (int b0 = c0; b0 < c1; b0 += 16) {
      float ps[16];
      int cs[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool in = b0 + i < c1;
        ps[i] = in ? part_p[size_t(b0 + i) * E + e] : 0.0f;
        cs[i] = in ? part_c[size_t(b0 + i) * E + e] : 0;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) { p += ps[i]; c += cs[i]; }
    }
    sp[threadIdx.x] = p;
    sc[threadIdx.x] = c;
  }
  __syncthreads();
  float term = 0.0f;
  if (int(threadIdx.x) < E) {
    float p = 0.0f;
    int c = 0;
    for (int i = 0; i < slices; ++i) { p += sp[i * E + threadIdx.x]; c += sc[i * E + threadIdx.x]; }
    counts[threadIdx.x] = c;
    term = float(c) * p;
  }
  term = warp_sum(term);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = term;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float sum = warp_sum(warp_sums[threadIdx.x]);
    if (threadIdx.x == 0) {
      *n_valid = n;
      *loss = n > 0 ? coef * float(E) / (float(n) * float(n) * float(k)) * sum : 0.0f;
    }
  }
}

// One warp per token; the row's gradient passes through shared memory, where
// the selected experts' own terms are added, one lane an expert (repeated ids
// add up first, in a fixed order).
template <int V, int NV>
__global__ void __launch_bounds__(kBalThreads, V * NV <= 16 ? 4 : 2)
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
  const int step = gridDim.x * kBalWarps;
  int t = blockIdx.x * kBalWarps + warp;
  // a token's logits are requested behind the token (or the counts) before it
  float next[NV * V] = {};
  bool live = t < T && (!valid || __ldg(valid + t));
  if (live && counts) load_logits<V, NV>(logits + t * ld, E, lane, next);
  float scale = 0.0f;
  if (counts) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) cf[e] = float(counts[e]);
    const float n = float(*n_valid);
    if (n > 0.0f) scale = (dloss ? *dloss : 1.0f) * coef * float(E) / (n * n * float(k));
  }
  __syncthreads();
  for (; t < T; t += step) {
    float g[NV * V];
    const bool now = live;
#pragma unroll
    for (int i = 0; i < NV * V; ++i) g[i] = next[i];
    float wj = 0.0f, dj = 0.0f;
    int id = 0;
    if (now && dw && lane < k) {
      wj = __ldg(w + size_t(t) * k + lane);
      dj = __ldg(dw + size_t(t) * k + lane);
      id = __ldg(ids + size_t(t) * k + lane);
    }
    live = t + step < T && (!valid || __ldg(valid + t + step));
    if (live && counts) load_logits<V, NV>(logits + (t + step) * ld, E, lane, next);
    if (now && counts) {
      row_exps(g);
      float z = 0.0f, zc = 0.0f, cv[NV * V];
      get_row<V, NV>(cf, E, lane, cv);
#pragma unroll
      for (int i = 0; i < NV * V; ++i) {
        z += g[i];
        zc = fmaf(g[i], cv[i], zc);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {   // the two sums side by side
        z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
        zc += __shfl_xor_sync(0xFFFFFFFFu, zc, off);
      }
      const float inv = inverse_sum(z), mean = zc * inv, f = scale * inv;
#pragma unroll
      for (int i = 0; i < NV * V; ++i) g[i] *= f * (cv[i] - mean);
    } else {
#pragma unroll
      for (int i = 0; i < NV * V; ++i) g[i] = 0.0f;
    }
    if (now && dw) {
      const float mine = wj * (dj - warp_sum(wj * dj));
      put_row<V, NV>(srow, E, lane, g);
      // the lowest lane of those with one id adds their terms, in lane order
      const bool sel = lane < k;
      if (sel && (id < 0 || id >= E)) set_device_status(FT_DEV_BAD_INDEX);
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, sel ? id : -1 - lane);
      float total = mine;
      if (__any_sync(0xFFFFFFFFu, __popc(peers) > 1)) {
        total = 0.0f;
        for (int j = 0; j < k; ++j) {
          const float add = __shfl_sync(0xFFFFFFFFu, mine, j);
          if (peers >> j & 1) total += add;
        }
      }
      __syncwarp();
      if (sel && id >= 0 && id < E && __ffs(peers) - 1 == lane) srow[id] += total;
      __syncwarp();
      get_row<V, NV>(srow, E, lane, g);
    }
    put_row<V, NV>(dlogits + t * ldd, E, lane, g);
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

// Clusters for T tokens: one of 8 warps a CTA, which needs no second launch, up
// to four tokens a warp (T = 256), else enough for a CTA of 16 warps a SM.  More
// of them cost more in sums than they hide, fewer warps hide less (8192 x 512,
// loss and gradient: 22.3 us; with 8 warps 23.9, two CTAs a SM 25.0, four 25.0;
// 64 x 128 in CTAs of 16 warps: 6.45 us instead of 6.25).
constexpr int kBalManyWarps = 16;
static int balance_clusters(int T, int num_sms) {
  if (T <= 4 * kBalWarps * kBalCluster) return 1;
  constexpr int per = kBalManyWarps * kBalCluster;
  return std::max(2, std::min((T + per - 1) / per, num_sms / kBalCluster));
}
static size_t balance_ws_bytes(int T, int E, int num_sms) {
  return size_t(balance_clusters(T, num_sms)) * (2 * size_t(E) + 1) * 4;
}

static cudaError_t launch_balance(const float* logits, long long ld, const int32_t* ids, const uint8_t* valid, int T,
                                  int E, int k, float coef, int32_t* counts, int32_t* n_valid, float* loss, void* ws,
                                  int num_sms, cudaStream_t s) {
  const int clusters = balance_clusters(T, num_sms);
  float* part_p = static_cast<float*>(ws);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + size_t(clusters) * E);
  int32_t* part_n = part_c + size_t(clusters) * E;
  const bool vec = E % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  const cudaError_t e = balance_variant(E, vec, [&](auto v, auto nv) {
    constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
    const bool one = clusters == 1;
    const int warps = one ? kBalWarps : kBalManyWarps;
    const size_t smem = ((warps + 1) * size_t(E) + warps + 4) * 4;
    auto kern = one ? balance_kernel<V, NV, kBalWarps> : balance_kernel<V, NV, kBalManyWarps>;
    if (smem > 48 * 1024) {
      const cudaError_t a = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
      if (a != cudaSuccess) return a;
    }
    ProfileScope prof(FT_KERNEL_BALANCE, s);
    return launch_pdl(kern, dim3(clusters * kBalCluster), dim3(32 * warps), smem, s, logits, ld, ids, valid, T, E, k,
                      coef, part_p, part_c, part_n, counts, n_valid, loss);
  });
  if (e != cudaSuccess || clusters == 1) return e;
  ProfileScope prof(FT_KERNEL_BALANCE, s);
  return launch_pdl(balance_finish_kernel, dim3(1), dim3(1024), 0, s, static_cast<const float*>(part_p),
                    static_cast<const int32_t*>(part_c), static_cast<const int32_t*>(part_n), clusters, E, k, coef,
                    counts, n_valid, loss);
}

static cudaError_t launch_route_backward(const float* logits, long long ld, const int32_t* ids, const float* w,
                                         const float* dw, const uint8_t* valid, int T, int E, int k, float coef,
                                         const int32_t* counts, const int32_t* n_valid, const float* dloss,
                                         float* dlogits, long long ldd, int num_sms, cudaStream_t s) {
  const bool vec = E % 4 == 0 && ld % 4 == 0 && ldd % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(dlogits) & 15) == 0;
  // four CTAs a SM, as many as fit (8192 x 512, loss and gradient: 22.3 us, with two 24.2, with eight in turns 22.8)
  const int blocks = int(std::min<long long>((T + kBalWarps - 1) / kBalWarps, 4LL * num_sms));
  return balance_variant(E, vec, [&](auto v, auto nv) {
    ProfileScope prof(FT_KERNEL_ROUTE_BACKWARD, s);
    return launch_pdl(route_backward_kernel<decltype(v)::value, decltype(nv)::value>, dim3(blocks), dim3(kBalThreads),
                      (kBalWarps + 1) * size_t(E) * 4, s, logits, ld, ids, w, dw, valid, T, E, k, coef, counts, n_valid,
                      dloss, dlogits, ldd);
  });
}

}  // namespace ftmoe
