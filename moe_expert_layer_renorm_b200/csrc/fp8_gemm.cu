// Products of E4M3 operands with fp32 block scales, on tcgen05 (kind::f8f6f4):
//   out[r, n] = sum_b sA[r, b] sB[n / 128, b] (sum_{k in block b} qA[r, k] qB[n, k])
// The inner sum of one 128-K block is four MMAs into a tensor-memory buffer
// that starts from zero; the epilogue warps read it back and add it, times the
// block's two scales, to fp32 accumulators in registers.  So the scales stay
// fp32 (they are not powers of two, which the MMA's own block scaling wants)
// and no sum inside the tensor core is longer than 128 terms.
//
// Two orientations:
//   few rows  (fp8_stream_kernel): the MMA's M side is 128 weight rows, its N
//     side up to BN token rows; bound by the weight bytes.  The grid's CTAs
//     share the K blocks of all output tiles evenly: each takes one contiguous
//     range of (tile, K block) pairs, and the partial sums of a tile that a
//     range border cuts are added by the last CTA to finish, in range order
//     (the same bits every time).
//   many rows (fp8_tile_kernel): the M side is 128 token rows, the N side 256
//     weight rows (256 output features; or 128 gate and 128 up rows of the same
//     features); a row's scales are one number a thread.
// Weights come by TMA from row-major codes [N, K] (3-D maps with the expert
// slot as the third coordinate), token rows as plain 2-D tiles; K past the end
// reads as zeros.
//
// Every pipeline wait is bounded as in ffn.cu.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sm100.cuh"

namespace ftmoe {

constexpr int kFp8WBytes = 128 * 128;   // 128 weight rows of one K block

struct Fp8Params {
  const float* sa;            // row scales [rows, nk], pitch ld_sa
  long long ld_sa;
  const float* sb[2];         // slot 0's weight scales [ceil(N/128), nk], pitch ld_sb
  long long ld_sb, slot_bytes;
  int nk;                     // K blocks
  int N;                      // output features
  const int4* units;          // grouped: {expert | slot << 10, feature tile, first row, rows}; null: dense
  const int* num_units;
  int rows, row_tiles, feat_tiles;   // dense
  void* out;                  // [rows, N], pitch ldo; for gate/up the codes of h
  int out_type;
  long long ldo;
  float* hs;                  // gate/up: scales of h [rows, ceil(N/128)]
  float* partials;            // stream kernel: two tiles for each CTA
  int* counters;              // stream kernel: arrivals at each cut tile, zero between launches
  int min_blocks;             // stream kernel: the fewest K blocks a CTA takes
};

struct Fp8Unit {
  int slot, ft, rb, nr;
};
// Unit u; dense units run over the row tiles of one feature tile first.
__device__ __forceinline__ Fp8Unit fp8_unit(const Fp8Params& p, int u, int bn) {
  if (p.units) {
    const int4 d = __ldg(p.units + u);
    return {d.x >> 10, d.y, d.z, d.w & 0xFFFF};
  }
  const int ft = u / p.row_tiles, rb = (u - ft * p.row_tiles) * bn;
  return {0, ft, rb, min(bn, p.rows - rb)};
}
__device__ __forceinline__ const float* fp8_weight_scales(const Fp8Params& p, int m, int slot, int block) {
  const uint8_t* base = reinterpret_cast<const uint8_t*>(p.sb[m]) + (long long)slot * p.slot_bytes;
  return reinterpret_cast<const float*>(base) + (long long)block * p.ld_sb;
}

// Instruction descriptor of kind::f8f6f4 with E4M3 operands and fp32 sums.
__host__ __device__ constexpr uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
      ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
// Each thread of the warp reads 32 consecutive 32-bit columns of its own lane.
__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
        "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
        "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
        "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr) : "memory");
}

// silu(g) u with the hardware exponential and a fast divide: a few fp32 steps
// (as the exponential overflows the quotient goes to 0, its limit).  One h a
// thread and column stands between a tile's last block and the next tile's
// first: with expf and two IEEE divisions here the gate/up kernel of 4096
// skewed tokens took 259 us instead of 176.
__device__ __forceinline__ float fp8_silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

__device__ __forceinline__ void store_as(void* out, int type, size_t i, float v) {
  if (type == FT_F32) static_cast<float*>(out)[i] = v;
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}
// |v| for a maximum that leaves NaN out, as ordered bits.
__device__ __forceinline__ uint32_t abs_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b > 0x7F800000u ? 0u : b;
}

// ---------------------------------------------------------- few rows ---

template <int NMAT, int BN>
struct Fp8StreamCfg {
  static constexpr int kStageBytes = NMAT * kFp8WBytes + BN * 128;
  static constexpr int kStages = 200 * 1024 / kStageBytes < 12 ? 200 * 1024 / kStageBytes : 12;
  static constexpr int kDB = 4;                        // accumulator buffers
  static constexpr int kTmemCols = kDB * NMAT * BN;    // a power of two, 64 .. 512
  static constexpr int kBars = 2 * kStages + 2 * kDB + 2;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kBars * 8 + 4 * BN * 4 + 32;
  static constexpr int kTileFloats = NMAT * BN * 128;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

constexpr int kFp8StreamThreads = 192;   // TMA warp, MMA warp, four epilogue warps
// One lane of a converged warp.  The MMA warps run their loops as a whole warp
// with warp-uniform values and issue inside this branch: descriptors and
// addresses then stay in uniform registers.  (Four MMAs of N = 32, their two
// commits and two passed waits take 333 cycles to issue this way, 528 from a
// loop of lane 0 alone -- more than the 512 the four MMAs of N = 256 run.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.b32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}

// Whether the phase is complete, without waiting for it.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
               " selp.b32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}

constexpr int kTagEpi = 9;               // barrier kind of a wait timeout: the epilogue warps' own barrier

// A barrier of the epilogue warps: an mbarrier, so that a warp that has given
// up leaves no other waiting without a limit.
struct EpiSync {
  uint64_t* bar;
  Abort ab;
  uint32_t phase;
  __device__ __forceinline__ bool sync(int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    const bool ok = __all_sync(0xFFFFFFFFu, ab.wait(bar, phase, kTagEpi));
    phase ^= 1;
    return ok;
  }
};

template <int NMAT, int BN>
__global__ void __launch_bounds__(kFp8StreamThreads, 1)
fp8_stream_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap tm_w0,
                  const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_rows) {
  using Cfg = Fp8StreamCfg<NMAT, BN>;
  constexpr int NST = Cfg::kStages, DB = Cfg::kDB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NST * Cfg::kStageBytes);
  uint64_t* empty = full + NST;
  uint64_t* d_full = empty + NST;
  uint64_t* d_empty = d_full + DB;
  uint64_t* drain_bar = d_empty + DB;
  uint64_t* epi_bar = drain_bar + 1;
  uint32_t* tmax = reinterpret_cast<uint32_t*>(epi_bar + 1);   // [4][BN]: each epilogue warp's maxima of h
  uint32_t* tmem_slot = tmax + 4 * BN;
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* last_flag = abort_flag + 1;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp-uniform
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < DB; ++i) { mbar_init(&d_full[i], 1); mbar_init(&d_empty[i], 4); }
    mbar_init(drain_bar, 1);
    mbar_init(epi_bar, 4);
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(&tm_w0);
    if (NMAT > 1) prefetch_tmap(&tm_w1);
    prefetch_tmap(&tm_rows);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, Cfg::kTmemCols); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const Abort ab{abort_flag};

  // this CTA's range of K blocks, all tiles' blocks in one line
  const int nk = p.nk;
  const long long total = (long long)(p.units ? *p.num_units : p.row_tiles * p.feat_tiles) * nk;
  const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)p.min_blocks);
  const long long g0 = min(total, per * blockIdx.x), g1 = min(total, g0 + per);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer ---
    if (lane == 0) {
      uint32_t i = 0;
      bool ok = true;
      int u = int(g0 / nk), kb = int(g0 - (long long)u * nk);
      for (long long g = g0; g < g1 && ok; ++u, kb = 0) {
        const Fp8Unit d = fp8_unit(p, u, BN);
        for (; kb < nk && g < g1; ++kb, ++g, ++i) {
          const int s = i % NST;
          if (!(ok = ab.wait(&empty[s], ((i / NST) & 1) ^ 1, kTagWEmpty, i, u))) break;
          uint8_t* dst = smem + s * Cfg::kStageBytes;
          mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
          tma_load_3d(dst, &tm_w0, &full[s], kb * 128, d.ft * 128, d.slot);
          if (NMAT > 1) tma_load_3d(dst + kFp8WBytes, &tm_w1, &full[s], kb * 128, d.ft * 128, d.slot);
          tma_load_2d(dst + NMAT * kFp8WBytes, &tm_rows, &full[s], kb * 128, d.rb);
        }
      }
      for (uint32_t j = (i > NST ? i - NST : 0); j < i; ++j) {   // drain: every copy has landed
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&full[j % NST], (j / NST) & 1) && globaltimer_ns() - t0 < 1000000000ull) {}
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer ---
    uint32_t i = 0;
    int s = 0, b = 0;
    bool ok = true;
    int u = int(g0 / nk), kb = int(g0 - (long long)u * nk);
    for (long long g = g0; g < g1 && ok; ++u, kb = 0) {
      const int n_eff = (fp8_unit(p, u, BN).nr + 15) & ~15;
      const uint32_t idesc = make_idesc_e4m3(128, n_eff);
      for (; kb < nk && g < g1; ++kb, ++g, ++i) {
        ok = ab.wait(&d_empty[b], ((i / DB) & 1) ^ 1, kTagDEmpty, i, u) &&
             ab.wait(&full[s], (i / NST) & 1, kTagWFull, i, u);
        if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
        tc_fence_after();
        if (elect_one()) {
          uint8_t* src = smem + s * Cfg::kStageBytes;
          const uint64_t rd = make_sdesc_sw128(smem_u32(src + NMAT * kFp8WBytes));
#pragma unroll
          for (int m = 0; m < NMAT; ++m) {
            const uint64_t wd = make_sdesc_sw128(smem_u32(src + m * kFp8WBytes));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_ss_f8(tmem + (b * NMAT + m) * BN, wd + 2 * j, rd + 2 * j, idesc, j > 0);
          }
          mma_commit(&empty[s]);
          mma_commit(&d_full[b]);
        }
        __syncwarp();
        if (++s == NST) s = 0;
        if (++b == DB) b = 0;
      }
    }
    if (i > 0) {   // drain: every MMA this warp issued has completed
      if (elect_one()) mma_commit(drain_bar);
      __syncwarp();
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < 1000000000ull) {}
    }
  } else {
    // ---------------------------------------------------- epilogue ---
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;                 // weight row within the tile = tensor-memory lane
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    constexpr int kGroups = (BN + 31) / 32;
    EpiSync epi{epi_bar, ab, 0};
    uint32_t i = 0;
    bool ok = true;
    const int u0 = int(g0 / nk);
    int u = u0, kb = int(g0 - (long long)u * nk);
    for (long long g = g0; g < g1; ++u, kb = 0) {
      const Fp8Unit d = fp8_unit(p, u, BN);
      const int n_eff = (d.nr + 15) & ~15;
      const bool whole = kb == 0 && g + nk <= g1;
      float acc[NMAT][BN];
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int n = 0; n < BN; ++n) acc[m][n] = 0.0f;
      const float* sw[NMAT];
#pragma unroll
      for (int m = 0; m < NMAT; ++m) sw[m] = fp8_weight_scales(p, m, d.slot, d.ft);
      for (; kb < nk && g < g1; ++kb, ++g, ++i) {
        float sr[kGroups], ws[NMAT];   // lane j of group q holds the scale of token row 32 q + j
#pragma unroll
        for (int q = 0; q < kGroups; ++q)
          sr[q] = q * 32 + lane < d.nr ? __ldg(p.sa + (d.rb + q * 32 + lane) * p.ld_sa + kb) : 0.0f;
#pragma unroll
        for (int m = 0; m < NMAT; ++m) ws[m] = __ldg(sw[m] + kb);
        const int b = i % DB;
        if (!(ok = __all_sync(0xFFFFFFFFu, ab.wait(&d_full[b], (i / DB) & 1, kTagDFull, i, u)))) break;
        tc_fence_after();
        const uint32_t dcol = tmem + lane_base + b * NMAT * BN;
#pragma unroll
        for (int c = 0; c < BN / 16; ++c) {
          if (c * 16 >= n_eff) break;
          uint32_t v[NMAT][16];
#pragma unroll
          for (int m = 0; m < NMAT; ++m) tmem_ld_32x32b_x16(dcol + m * BN + c * 16, v[m]);
          tmem_wait_ld();
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const float s = __shfl_sync(0xFFFFFFFFu, sr[c / 2], (c & 1) * 16 + n);
#pragma unroll
            for (int m = 0; m < NMAT; ++m)
              acc[m][c * 16 + n] = fmaf(__uint_as_float(v[m][n]), s * ws[m], acc[m][c * 16 + n]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[b]);
      }
      if (!ok) break;
      if (!whole) {
        // a cut tile: leave the partial sums, and the last CTA to arrive adds them all up in range order
        float* mine = p.partials + ((long long)blockIdx.x * 2 + (u != u0)) * Cfg::kTileFloats + row;
#pragma unroll
        for (int m = 0; m < NMAT; ++m)
#pragma unroll
          for (int n = 0; n < BN; ++n)
            if (n < d.nr) __stcg(mine + (m * BN + n) * 128, acc[m][n]);
        const long long first = (long long)u * nk / per, end = ((long long)(u + 1) * nk - 1) / per;
        __threadfence();
        if (!(ok = epi.sync(lane))) break;
        if (threadIdx.x == 64) *last_flag = atomicAdd(p.counters + u, 1) == int(end - first);
        if (!(ok = epi.sync(lane))) break;
        if (!*last_flag) continue;
        __threadfence();
        if (threadIdx.x == 64) p.counters[u] = 0;
#pragma unroll
        for (int m = 0; m < NMAT; ++m)
#pragma unroll
          for (int n = 0; n < BN; ++n) acc[m][n] = 0.0f;
        for (long long c = first; c <= end; ++c) {
          // CTA c's first tile unless its range began in an earlier one
          const bool second = c * per / nk != u;
          const float* part = p.partials + (c * 2 + second) * Cfg::kTileFloats + row;
#pragma unroll
          for (int m = 0; m < NMAT; ++m)
#pragma unroll
            for (int n = 0; n < BN; ++n)
              if (n < d.nr) acc[m][n] += __ldcg(part + (m * BN + n) * 128);
        }
      }
      const int feat = d.ft * 128 + row;
      if constexpr (NMAT == 1) {
        if (feat < p.N) {
#pragma unroll
          for (int n = 0; n < BN; ++n)
            if (n < d.nr) store_as(p.out, p.out_type, (d.rb + n) * p.ldo + feat, acc[0][n]);
        }
      } else {
        // h = silu(gate) up; its scale is the maximum over the tile's 128 features (those past N are zeros)
#pragma unroll
        for (int n = 0; n < BN; ++n) {
          if (n >= d.nr) break;
          acc[0][n] = fp8_silu_mul(acc[0][n], acc[NMAT - 1][n]);
          const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, abs_bits(acc[0][n]));
          if (lane == 0) tmax[quarter * BN + n] = m;
        }
        if (!(ok = epi.sync(lane))) break;
        uint8_t* h = static_cast<uint8_t*>(p.out);
        const int hb = (p.N + kFp8Block - 1) / kFp8Block;
#pragma unroll
        for (int n = 0; n < BN; ++n) {
          if (n >= d.nr) break;
          const uint32_t m = max(max(tmax[n], tmax[BN + n]), max(tmax[2 * BN + n], tmax[3 * BN + n]));
          const Fp8Scale f = fp8_scale_of(__uint_as_float(m));
          if (feat < p.N) h[(d.rb + n) * p.ldo + feat] = uint8_t(cvt_e4m3x2(acc[0][n] * fp8_factor_of(f), 0.0f));
          if (row == 0) p.hs[(long long)(d.rb + n) * hb + d.ft] = f.scale;
        }
        if (!(ok = epi.sync(lane))) break;   // the maxima are read before the next tile's are written
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// --------------------------------------------------------- many rows ---

constexpr int kFp8TileThreads = 384;   // TMA warp, MMA warp, two idle; two epilogue warpgroups
constexpr int kFp8TileStages = 4;
constexpr int kFp8TileStageBytes = 3 * 128 * 128;
constexpr int kFp8TileOutBytes = 8 * 4096;   // output staging of the eight epilogue warps; for gate/up the row maxima
constexpr int kFp8TileSmemBytes =
    1024 + kFp8TileStages * kFp8TileStageBytes + kFp8TileOutBytes + (2 * kFp8TileStages + 6) * 8 + 32;

__device__ __forceinline__ unsigned long long pack2(uint32_t lo, uint32_t hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ void fma2(unsigned long long& acc, unsigned long long a, unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

template <int NMAT>
__global__ void __launch_bounds__(kFp8TileThreads, 1)
fp8_tile_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap tm_w0,
                const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_rows) {
  constexpr int NST = kFp8TileStages, DB = 2;   // DB: accumulator buffers
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_stage = smem + NST * kFp8TileStageBytes;
  uint32_t* tmax = reinterpret_cast<uint32_t*>(out_stage);   // [unit parity][half][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(out_stage + kFp8TileOutBytes);
  uint64_t* empty = full + NST;
  uint64_t* d_full = empty + NST;
  uint64_t* d_empty = d_full + DB;
  uint64_t* drain_bar = d_empty + DB;
  uint64_t* epi_bar = drain_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(epi_bar + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp-uniform
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < DB; ++i) { mbar_init(&d_full[i], 1); mbar_init(&d_empty[i], 8); }
    mbar_init(drain_bar, 1);
    mbar_init(epi_bar, 8);
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(&tm_w0);
    if (NMAT > 1) prefetch_tmap(&tm_w1);
    prefetch_tmap(&tm_rows);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const Abort ab{abort_flag};
  const int nk = p.nk;
  const int n_units = p.units ? *p.num_units : p.row_tiles * p.feat_tiles;

  // registers: 384 threads x 168 at launch = 128 x 56 + 256 x 224
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------------------------------------- TMA producer ---
      if (lane == 0) {
        uint32_t i = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
          const Fp8Unit d = fp8_unit(p, u, 128);
          for (int kb = 0; kb < nk; ++kb, ++i) {
            const int s = i % NST;
            if (!(ok = ab.wait(&empty[s], ((i / NST) & 1) ^ 1, kTagWEmpty, i, u))) break;
            uint8_t* dst = smem + s * kFp8TileStageBytes;
            mbar_arrive_expect_tx(&full[s], kFp8TileStageBytes);
            tma_load_2d(dst, &tm_rows, &full[s], kb * 128, d.rb);
            uint8_t* wdst = dst + kFp8WBytes;
            if (NMAT == 2) {   // each half: 64 gate rows, then the up rows of the same 64 features
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                tma_load_3d(wdst + h * kFp8WBytes, &tm_w0, &full[s], kb * 128, d.ft * 128 + h * 64, d.slot);
                tma_load_3d(wdst + h * kFp8WBytes + kFp8WBytes / 2, &tm_w1, &full[s], kb * 128, d.ft * 128 + h * 64, d.slot);
              }
            } else {           // one box of 256 rows
              tma_load_3d(wdst, &tm_w0, &full[s], kb * 128, d.ft * 256, d.slot);
            }
          }
        }
        for (uint32_t j = (i > NST ? i - NST : 0); j < i; ++j) {   // drain
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(&full[j % NST], (j / NST) & 1) && globaltimer_ns() - t0 < 1000000000ull) {}
        }
      }
    } else if (warp == 1) {
      // ----------------------------------------------- MMA issuer ---
      // The barriers of the next block are tried right after this block's MMAs
      // are issued, both at once: a try_wait takes some 85 cycles to answer
      // even when its phase is complete.
      constexpr uint32_t idesc = make_idesc_e4m3(128, 256);
      uint32_t i = 0;
      int s = 0, b = 0;
      bool ok = true, tried = false, have_rows = false, have_d = false;
      for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
        for (int kb = 0; kb < nk; ++kb, ++i) {
          if (!tried || !have_rows) ok = ab.wait(&full[s], (i / NST) & 1, kTagWFull, i, u);
          if (!tried || !have_d) ok = ok && ab.wait(&d_empty[b], ((i / DB) & 1) ^ 1, kTagDEmpty, i, u);
          if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t rd = make_sdesc_sw128(smem_u32(smem + s * kFp8TileStageBytes));
            const uint64_t wd = make_sdesc_sw128(smem_u32(smem + s * kFp8TileStageBytes + kFp8WBytes));
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_ss_f8(tmem + b * 256, rd + 2 * j, wd + 2 * j, idesc, j > 0);
            mma_commit(&d_full[b]);
            mma_commit(&empty[s]);
          }
          __syncwarp();
          if (++s == NST) s = 0;
          b ^= 1;
          have_rows = mbar_test_wait(&full[s], ((i + 1) / NST) & 1);
          have_d = mbar_test_wait(&d_empty[b], (((i + 1) / DB) & 1) ^ 1);
          tried = true;
        }
      }
      if (i > 0) {   // drain
        if (elect_one()) mma_commit(drain_bar);
        __syncwarp();
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < 1000000000ull) {}
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // -------------------------------------------------- epilogue ---
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;                 // token row within the tile = tensor-memory lane
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    EpiSync epi{epi_bar, ab, 0};
    uint32_t i = 0;
    bool ok = true;
    int parity = 0;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x, parity ^= 1) {
      const Fp8Unit d = fp8_unit(p, u, 128);
      const bool live = row < d.nr;
      const float* sr = p.sa + (long long)(d.rb + (live ? row : 0)) * p.ld_sa;
      // a feature block past the end has no scales: its columns are zeros, and block 0's scale does
      const int block = NMAT == 2 ? d.ft : d.ft * 2 + half;
      const bool has = block * kFp8Block < p.N;
      const float* sw0 = fp8_weight_scales(p, 0, d.slot, has ? block : 0);
      const float* sw1 = NMAT == 2 ? fp8_weight_scales(p, 1, d.slot, block) : sw0;
      unsigned long long acc[64];   // NMAT 1: 128 columns; NMAT 2: gate of 64 features, then up
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0ull;
      float a = __ldg(sr), w0 = __ldg(sw0), w1 = NMAT == 2 ? __ldg(sw1) : 0.0f;
      // Chunks of 32 columns in two register buffers, the next chunk's load in
      // flight behind one chunk's sums -- also across blocks: the last chunk's
      // sums stand behind the next block's first load.
      uint32_t v[2][32];
      if (!(ok = __all_sync(0xFFFFFFFFu, ab.wait(&d_full[i & 1], (i >> 1) & 1, kTagDFull, i, u)))) break;
      tc_fence_after();
      const uint32_t dcol = tmem + lane_base + half * 128;
      tmem_ld_32x32b_x32(dcol + (i & 1) * 256, v[0]);
      for (int kb = 0; kb < nk; ++kb, ++i) {
        const uint32_t b = i & 1;
        const float s0 = a * w0, s1 = a * w1;
        const unsigned long long p0 = pack2(__float_as_uint(s0), __float_as_uint(s0));
        const unsigned long long p1 = NMAT == 2 ? pack2(__float_as_uint(s1), __float_as_uint(s1)) : p0;
        const bool more = kb + 1 < nk;
        if (more) {
          a = __ldg(++sr);
          w0 = __ldg(++sw0);
          if (NMAT == 2) w1 = __ldg(++sw1);
        }
        bool ready = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_wait_ld();
          if (c < 3) {
            tmem_ld_32x32b_x32(dcol + b * 256 + (c + 1) * 32, v[(c + 1) & 1]);
            if (c == 1) ready = mbar_test_wait(&d_full[b ^ 1], ((i + 1) >> 1) & 1);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[b]);
            if (more) {
              if (!ready) ok = ab.wait(&d_full[b ^ 1], ((i + 1) >> 1) & 1, kTagDFull, i + 1, u);
              if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
              tc_fence_after();
              tmem_ld_32x32b_x32(dcol + (b ^ 1) * 256, v[0]);
            }
          }
#pragma unroll
          for (int n = 0; n < 16; ++n) fma2(acc[c * 16 + n], pack2(v[c & 1][2 * n], v[c & 1][2 * n + 1]), c < 2 ? p0 : p1);
        }
        if (!ok) break;
      }
      if (!ok) break;
      if constexpr (NMAT == 1) {
        // Through 4 KB of shared memory a warp, 64 bf16 or 32 fp32 columns of its
        // 32 rows at a time: a thread has a row's columns, but stores of whole
        // 128-byte rows, four rows an instruction, are what the memory takes
        // well (16-byte stores to 32 rows took half of the unit's time).
        uint8_t* stage = out_stage + (warp - 4) * 4096;
        const int f0 = d.ft * 256 + half * 128;
        const int esize = p.out_type == FT_F32 ? 4 : 2;
        const bool vec = (p.ldo * esize) % 16 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 32) {
          // 16-byte piece q of the thread's row at q ^ (row % 8)
          const bool f32 = p.out_type == FT_F32;
          if (f32) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float2 x = unpack2(acc[c0 / 2 + 2 * q]), y = unpack2(acc[c0 / 2 + 2 * q + 1]);
              *reinterpret_cast<float4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = make_float4(x.x, x.y, y.x, y.y);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 x = unpack2(acc[c0 / 2 + 4 * q + e]);
                const __nv_bfloat162 t = __floats2bfloat162_rn(x.x, x.y);
                o[e] = *reinterpret_cast<const uint32_t*>(&t);
              }
              const int piece = (c0 & 32) / 8 + q;
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((piece ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (!(c0 & 32)) continue;
          }
          __syncwarp();
          const int fc = f0 + (f32 ? c0 : c0 - 32);   // the chunk's first feature
#pragma unroll
          for (int r = 0; r < 32; r += 4) {
            const int rr = r + (lane >> 3), piece = lane & 7;
            const uint4 x = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((piece ^ (rr & 7)) << 4));
            const int tile_row = quarter * 32 + rr, f = fc + piece * (16 / esize);
            if (tile_row >= d.nr || f >= p.N) continue;
            uint8_t* dst = static_cast<uint8_t*>(p.out) + ((d.rb + tile_row) * p.ldo + f) * esize;
            if (vec && f + 16 / esize <= p.N) {
              *reinterpret_cast<uint4*>(dst) = x;
            } else {
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if (f32) {
                  if (e < 4 && f + e < p.N) reinterpret_cast<uint32_t*>(dst)[e] = w[e & 3];
                } else if (f + e < p.N) {
                  reinterpret_cast<uint16_t*>(dst)[e] = uint16_t(w[e / 2] >> (16 * (e & 1)));
                }
              }
            }
          }
          __syncwarp();
        }
      } else {
        // h of this thread's 64 features; its scale is the maximum over the row's 128 (those past N are zeros)
        float h[64];
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 g = unpack2(acc[c]), up = unpack2(acc[32 + c]);
          h[2 * c] = fp8_silu_mul(g.x, up.x);
          h[2 * c + 1] = fp8_silu_mul(g.y, up.y);
          m = max(m, max(abs_bits(h[2 * c]), abs_bits(h[2 * c + 1])));
        }
        tmax[parity * 256 + half * 128 + row] = m;
        if (!(ok = epi.sync(lane))) break;
        m = max(m, tmax[parity * 256 + (half ^ 1) * 128 + row]);
        const Fp8Scale f = fp8_scale_of(__uint_as_float(m));
        const float inv = fp8_factor_of(f);
        const int f0 = d.ft * 128 + half * 64;
        if (live) {
          if (half == 0) p.hs[(long long)(d.rb + row) * ((p.N + kFp8Block - 1) / kFp8Block) + d.ft] = f.scale;
          if (f0 < p.N) {   // N is a multiple of 64
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (d.rb + row) * p.ldo + f0);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t o[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                o[q] = cvt_e4m3x2(h[16 * c + 4 * q] * inv, h[16 * c + 4 * q + 1] * inv) |
                       (cvt_e4m3x2(h[16 * c + 4 * q + 2] * inv, h[16 * c + 4 * q + 3] * inv) << 16);
              dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------ prep kernels ---

__global__ void __launch_bounds__(256) fp8_zero_kernel(int* counters, int n) {
  pdl_enter();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) counters[i] = 0;
}

// One launch: blocks [0, sched.nsched) build the two work lists and clear the
// counters (prep_schedule of ffn.cu), the others write the token rows in FP8
// in permuted order, sixteen lanes a group of 128 values.
struct Fp8PrepParams {
  PrepParams sched;
  const __nv_bfloat16* x;
  int T;
  uint8_t* codes;
  float* scales;
};
__global__ void __launch_bounds__(256) fp8_prep_kernel(const Fp8PrepParams p) {
  pdl_enter();
  if (int(blockIdx.x) < p.sched.nsched) {
    prep_schedule(p.sched, blockIdx.x);
    return;
  }
  const int H = p.sched.H, nb = (H + kFp8Block - 1) / kFp8Block;
  const long long g = ((long long)(blockIdx.x - p.sched.nsched) * blockDim.x + threadIdx.x) >> 4;
  const bool live = g < (long long)p.sched.P * nb;
  const int sub = threadIdx.x & 15;
  const int r = live ? int(g / nb) : 0;
  const int b = live ? int(g - (long long)r * nb) : 0;
  const int src = __ldg(p.sched.perm_src + r);
  const int t = src / p.sched.k_top;
  const bool known = src >= 0 && t < p.T;
  if (live && !known && b == 0 && sub == 0) set_device_status(FT_DEV_BAD_INDEX);
  const int k0 = b * kFp8Block + sub * 8;
  float v[8];
  load8<__nv_bfloat16, true>(p.x + (long long)(known ? t : 0) * H + k0, live && known ? min(8, H - k0) : 0, v);
  float m = absmax8(v);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  if (!live) return;
  const Fp8Scale f = fp8_scale_of(m);
  if (sub == 0) p.scales[(long long)r * nb + b] = f.scale;
  if (k0 < H)   // H is a multiple of 64
    *reinterpret_cast<uint2*>(p.codes + (long long)r * H + k0) =
        make_uint2(fp8_codes4(v[0], v[1], v[2], v[3], f), fp8_codes4(v[4], v[5], v[6], v[7], f));
}

// ---------------------------------------------------------------- host ---

// Codes [rows, K] (pitch bytes) as boxes of 128 K x box_rows, 128-byte swizzle.
static bool make_fp8_map(const void* base, long long rows, int K, long long pitch, int slots, long long slot_bytes,
                         int box_rows, bool three_d, CUtensorMap* m) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cuuint64_t(K), cuuint64_t(rows), cuuint64_t(slots)};
  const cuuint64_t strides[2] = {cuuint64_t(pitch), cuuint64_t(slot_bytes)};
  const cuuint32_t box[3] = {128, cuuint32_t(box_rows), 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, three_d ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch with the kernel's dynamic shared memory allowed on the current device.
template <typename... KArgs, typename... Args>
static cudaError_t launch_fp8(void (*kern)(KArgs...), int grid, int threads, int smem, std::atomic<uint64_t>& done,
                              cudaStream_t s, Args&&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(done.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(uint64_t(1) << dev);
  }
  return launch_pdl(kern, dim3(grid), dim3(threads), smem, s, std::forward<Args>(args)...);
}
template <int NMAT, int BN>
static cudaError_t launch_fp8_stream(const Fp8Params& p, int grid, const CUtensorMap& w0, const CUtensorMap& w1,
                                     const CUtensorMap& rows, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  return launch_fp8(fp8_stream_kernel<NMAT, BN>, grid, kFp8StreamThreads, Fp8StreamCfg<NMAT, BN>::kSmemBytes, done, s, p,
                    w0, w1, rows);
}
template <int NMAT>
static cudaError_t launch_fp8_tile(const Fp8Params& p, int grid, const CUtensorMap& w0, const CUtensorMap& w1,
                                   const CUtensorMap& rows, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  return launch_fp8(fp8_tile_kernel<NMAT>, grid, kFp8TileThreads, kFp8TileSmemBytes, done, s, p, w0, w1, rows);
}
template <int NMAT>
static cudaError_t launch_fp8_any(int bn, const Fp8Params& p, int grid, const CUtensorMap& w0, const CUtensorMap& w1,
                                  const CUtensorMap& rows, cudaStream_t s) {
  switch (bn) {
    case 16: return launch_fp8_stream<NMAT, 16>(p, grid, w0, w1, rows, s);
    case 32: return launch_fp8_stream<NMAT, 32>(p, grid, w0, w1, rows, s);
    case 64: return launch_fp8_stream<NMAT, 64>(p, grid, w0, w1, rows, s);
    default: return launch_fp8_tile<NMAT>(p, grid, w0, w1, rows, s);
  }
}

// Token rows a tile takes (16, 32, 64: the stream kernel; 128: the tile kernel).
static int fp8_rows_tile(double rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

struct Fp8GemmPlan {
  int bn, row_tiles, feat_tiles, grid, min_blocks;
  bool cut;            // a tile may be cut between CTAs
  size_t off_part, total;
};
static Fp8GemmPlan plan_fp8_gemm(int M, int N, int K, int num_sms) {
  Fp8GemmPlan pl{};
  const int nk = fp8_blocks(K);
  const long long big = ((M + 127LL) / 128) * ((N + 255LL) / 256);
  pl.bn = M <= 64 ? fp8_rows_tile(M) : big * 2 >= num_sms ? 128 : 64;
  pl.row_tiles = (M + pl.bn - 1) / pl.bn;
  pl.feat_tiles = pl.bn == 128 ? (N + 255) / 256 : (N + 127) / 128;
  const long long units = (long long)pl.row_tiles * pl.feat_tiles;
  pl.min_blocks = 1;
  if (pl.bn == 128) {
    pl.grid = int(std::min<long long>(units, num_sms));
    return pl;
  }
  const long long per = std::max<long long>((units * nk + num_sms - 1) / num_sms, pl.min_blocks);
  pl.grid = int((units * nk + per - 1) / per);
  pl.cut = per % nk != 0;
  if (pl.cut) {
    pl.off_part = align256(size_t(units) * 4);
    pl.total = pl.off_part + size_t(pl.grid) * 2 * pl.bn * 128 * 4;
  }
  return pl;
}
static size_t fp8_gemm_ws_bytes(int M, int N, int K) { return plan_fp8_gemm(M, N, K, device_sm_count()).total; }

static cudaError_t launch_fp8_gemm(const uint8_t* a, long long lda, const float* sa, long long ld_sa, const uint8_t* b,
                                   long long ldb, const float* sb, long long ld_sb, int M, int N, int K, void* out,
                                   int out_type, long long ldo, void* ws, cudaStream_t s, const char** why) {
  const Fp8GemmPlan pl = plan_fp8_gemm(M, N, K, device_sm_count());
  CUtensorMap tm_a, tm_b;
  if (!make_fp8_map(a, M, K, lda, 1, 16, pl.bn, false, &tm_a) ||
      !make_fp8_map(b, N, K, ldb, 1, ldb * N, pl.bn == 128 ? 256 : 128, true, &tm_b)) {
    *why = "ft_fp8_gemm: cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  Fp8Params p{};
  p.sa = sa;
  p.ld_sa = ld_sa;
  p.sb[0] = p.sb[1] = sb;
  p.ld_sb = ld_sb;
  p.nk = fp8_blocks(K);
  p.N = N;
  p.rows = M;
  p.row_tiles = pl.row_tiles;
  p.feat_tiles = pl.feat_tiles;
  p.out = out;
  p.out_type = out_type;
  p.ldo = ldo;
  p.min_blocks = pl.min_blocks;
  if (pl.cut) {
    p.counters = static_cast<int*>(ws);
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + pl.off_part);
    const int n = pl.row_tiles * pl.feat_tiles;
    ProfileScope prof(FT_KERNEL_FP8_GEMM, s);
    const cudaError_t e = launch_pdl(fp8_zero_kernel, dim3(std::min(32, (n + 255) / 256)), dim3(256), 0, s, p.counters, n);
    if (e != cudaSuccess) return e;
  }
  ProfileScope prof(FT_KERNEL_FP8_GEMM, s);
  return launch_fp8_any<1>(pl.bn, p, pl.grid, tm_b, tm_b, tm_a, s);
}

struct Fp8FfnPlan {
  int bn, mt1, mt2;                 // token rows a tile takes; feature tiles of gate/up and down
  long long max_units1, max_units2;
  int grid1, grid2;
  size_t off_x, off_xs, off_h, off_hs, off_units1, off_units2, off_counts, off_cnt1, off_cnt2, off_part, total;
};
static Fp8FfnPlan plan_fp8_ffn(int T, int H, int I, int E, int k) {
  Fp8FfnPlan p{};
  const int num_sms = device_sm_count();
  const long long P = (long long)T * k;
  const double distinct = E * (1.0 - pow(1.0 - double(k) / E, double(T)));
  // a quarter more than the mean, so that most groups of an even spread are one tile
  p.bn = fp8_rows_tile(1.25 * double(P) / std::max(distinct, 1.0));
  p.mt1 = fp8_blocks(I);
  p.mt2 = p.bn == 128 ? (H + 255) / 256 : fp8_blocks(H);
  const long long tiles = std::min<long long>(E, P) + P / p.bn;
  p.max_units1 = tiles * p.mt1;
  p.max_units2 = tiles * p.mt2;
  const bool stream = p.bn < 128;
  p.grid1 = stream ? num_sms : int(std::min<long long>(num_sms, p.max_units1));
  p.grid2 = stream ? num_sms : int(std::min<long long>(num_sms, p.max_units2));
  size_t o = 0;
  p.off_x = o;      o = align256(o + size_t(P) * H);
  p.off_xs = o;     o = align256(o + size_t(P) * fp8_blocks(H) * 4);
  p.off_h = o;      o = align256(o + size_t(P) * I);
  p.off_hs = o;     o = align256(o + size_t(P) * fp8_blocks(I) * 4);
  p.off_units1 = o; o = align256(o + size_t(p.max_units1) * 16);
  p.off_units2 = o; o = align256(o + size_t(p.max_units2) * 16);
  p.off_counts = o; o = align256(o + 16);
  p.off_cnt1 = o;   o = align256(o + (stream ? size_t(p.max_units1) * 4 : 0));
  p.off_cnt2 = o;   o = align256(o + (stream ? size_t(p.max_units2) * 4 : 0));
  p.off_part = o;   o = align256(o + (stream ? size_t(num_sms) * 2 * 2 * p.bn * 128 * 4 : 0));
  p.total = o;
  return p;
}

static cudaError_t launch_fp8_ffn(const void* x, int T, int H, int I, int E, int k, const int32_t* perm_src,
                                  const int32_t* offsets, const int32_t* slot_table, const void* pool_v,
                                  const ft_nvfp4_slot_layout& L, void* out, int out_type, void* ws, cudaStream_t s,
                                  const char** why) {
  const Fp8FfnPlan pl = plan_fp8_ffn(T, H, I, E, k);
  const uint8_t* pool = static_cast<const uint8_t*>(pool_v);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int P = T * k;
  const bool stream = pl.bn < 128;
  CUtensorMap tm[3], tm_x, tm_h;
  const int rows[3] = {I, I, H}, Ks[3] = {H, H, I};
  bool ok = make_fp8_map(w + pl.off_x, P, H, H, 1, 16, pl.bn, false, &tm_x) &&
            make_fp8_map(w + pl.off_h, P, I, I, 1, 16, pl.bn, false, &tm_h);
  for (int m = 0; m < 3; ++m)
    ok = ok && make_fp8_map(pool + L.codes_off[m], rows[m], Ks[m], Ks[m], L.num_slots, L.slot_bytes,
                            stream ? 128 : m == FT_DOWN ? 256 : 64, true, &tm[m]);
  if (!ok) {
    *why = "ft_moe_ffn_fp8: cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  int4* units1 = reinterpret_cast<int4*>(w + pl.off_units1);
  int4* units2 = reinterpret_cast<int4*>(w + pl.off_units2);
  int* counts = reinterpret_cast<int*>(w + pl.off_counts);
  cudaError_t e;
  {
    Fp8PrepParams pp{};
    PrepParams& sp = pp.sched;
    sp.offsets = offsets;
    sp.slot_table = slot_table;
    sp.E = E;
    sp.num_slots = L.num_slots;
    sp.nsched = int(std::min<long long>(32, std::max<long long>(1, (pl.max_units1 + pl.max_units2) / 4096)));
    sp.bn1 = sp.bn2 = pl.bn;
    sp.mt1 = pl.mt1;
    sp.mt2 = pl.mt2;
    sp.s1 = sp.s2 = 1;
    sp.units1 = units1;
    sp.units2 = units2;
    sp.counts = counts;
    sp.counters1 = reinterpret_cast<int*>(w + pl.off_cnt1);
    sp.ncnt1 = stream ? int(pl.max_units1) : 0;
    sp.counters2 = reinterpret_cast<int*>(w + pl.off_cnt2);
    sp.ncnt2 = stream ? int(pl.max_units2) : 0;
    sp.perm_src = perm_src;
    sp.P = P;
    sp.k_top = k;
    sp.H = H;
    pp.x = static_cast<const __nv_bfloat16*>(x);
    pp.T = T;
    pp.codes = w + pl.off_x;
    pp.scales = reinterpret_cast<float*>(w + pl.off_xs);
    const long long threads = 16LL * P * fp8_blocks(H);
    ProfileScope prof(FT_KERNEL_PREP, s);
    e = launch_pdl(fp8_prep_kernel, dim3(unsigned(sp.nsched + (threads + 255) / 256)), dim3(256), 0, s, pp);
  }
  if (e != cudaSuccess) return e;
  Fp8Params p{};
  p.sa = reinterpret_cast<const float*>(w + pl.off_xs);
  p.ld_sa = fp8_blocks(H);
  for (int m = 0; m < 2; ++m) p.sb[m] = reinterpret_cast<const float*>(pool + L.scales_off[m]);
  p.ld_sb = L.ld_scale[FT_GATE] / 4;
  p.slot_bytes = L.slot_bytes;
  p.nk = fp8_blocks(H);
  p.N = I;
  p.units = units1;
  p.num_units = counts;
  p.out = w + pl.off_h;
  p.ldo = I;
  p.hs = reinterpret_cast<float*>(w + pl.off_hs);
  p.partials = reinterpret_cast<float*>(w + pl.off_part);
  p.counters = reinterpret_cast<int*>(w + pl.off_cnt1);
  p.min_blocks = 1;
  {
    ProfileScope prof(FT_KERNEL_FP8_GATE_UP, s);
    e = launch_fp8_any<2>(pl.bn, p, pl.grid1, tm[FT_GATE], tm[FT_UP], tm_x, s);
  }
  if (e != cudaSuccess) return e;
  p.sa = reinterpret_cast<const float*>(w + pl.off_hs);
  p.ld_sa = fp8_blocks(I);
  p.sb[0] = p.sb[1] = reinterpret_cast<const float*>(pool + L.scales_off[FT_DOWN]);
  p.ld_sb = L.ld_scale[FT_DOWN] / 4;
  p.nk = fp8_blocks(I);
  p.N = H;
  p.units = units2;
  p.num_units = counts + 1;
  p.out = out;
  p.out_type = out_type;
  p.ldo = H;
  p.counters = reinterpret_cast<int*>(w + pl.off_cnt2);
  ProfileScope prof(FT_KERNEL_FP8_DOWN, s);
  return launch_fp8_any<1>(pl.bn, p, pl.grid2, tm[FT_DOWN], tm[FT_DOWN], tm_h, s);
}

}  // namespace ftmoe
