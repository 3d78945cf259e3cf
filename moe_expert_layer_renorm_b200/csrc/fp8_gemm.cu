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
//     form clusters of 1, 2, 4 or 8 that share a tile's K blocks; the partial
//     sums meet through distributed shared memory and are added in the order
//     of the cluster's ranks (the same bits every time).
//   many rows (fp8_tile_kernel): the M side is 128 token rows, the N side 256
//     weight rows (256 output features; or 128 gate and 128 up rows of the same
//     features); a row's scales are one number a thread.
// Weights come by TMA from row-major codes [N, K] (3-D maps with the expert
// slot as the third coordinate), token rows as plain 2-D tiles; K past the end
// reads as zeros.
//
// Every pipeline wait is bounded as in ffn.cu.
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "cluster.cuh"
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
  // stream kernel
  const int32_t* offsets;     // grouped: group offsets [E + 1] and slots [E]; null: dense
  const int32_t* slot_table;
  int E, num_slots;
  int split;                  // CTAs (one cluster) that share a tile's K blocks
  int early;                  // weights and groups are older than the kernel before this one
  int share;                  // host: the kernels that share a SM
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

__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[32]) { tmem_ld_32x32b_x32(taddr, v); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[16]) { tmem_ld_32x32b_x16(taddr, v); }

// silu(g) u, as g s u with s = (g >= 0 ? 1 : e) / (1 + e) and e = e^-|g|: nothing
// overflows, whatever g, and the divisor lies in [1, 2], so that an approximate
// reciprocal and one remainder step (as quotient_by) give the quotient to a step
// or two of fp32.  A non-finite g follows g / (1 + e^-g): e is 0 or NaN.
// One h a thread and column stands between a tile's last block and the next
// tile's first.  The hardware exponential and a fast divide would save 6 us of
// 282 of the FFN (4096 skewed tokens, 2048 x 768, 128 experts, k = 8), but lose up
// to 2^-18 of h, and all of it where 1 + e^-g passes 2^126.
__device__ __forceinline__ float fp8_silu_mul(float g, float u) {
  const float e = expf(-fabsf(g)), d = 1.0f + e;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return g * quotient_by(g >= 0.0f ? 1.0f : e, d, r) * u;
}

// |v| for a maximum that leaves NaN out, as ordered bits.
__device__ __forceinline__ uint32_t abs_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b > 0x7F800000u ? 0u : b;
}

// ---------------------------------------------------------- few rows ---

// SHARE: gate/up and down leave each other room on a SM, so that the down
// kernel's first weights are on their way while gate/up still runs (one set of
// epilogue warps, 3 or 4 stages, 8 accumulator buffers).
template <int NMAT, int BN, bool SHARE>
struct Fp8StreamCfg {
  // Two sets of four epilogue warps take turns at the tiles where registers allow: a down tile of 6 blocks is finished
  // in some 7000 cycles, longer than its weights take to arrive.
  static constexpr int kSets = NMAT * BN <= 64 && !SHARE ? 2 : 1;
  static constexpr int kThreads = 64 + 128 * kSets;             // TMA warp, MMA warp, epilogue warps
  static constexpr int kStageBytes = NMAT * kFp8WBytes + BN * 128;
  // partial sums from the other CTAs of the cluster; none where they would take more than 32 KB
  static constexpr int kXBytes = NMAT * BN * 512 <= 32768 ? NMAT * BN * 512 : 0;
  static constexpr int kStages = SHARE ? (NMAT == 2 ? 4 : 3) : (208 * 1024 - kXBytes) / kStageBytes;
  // accumulator buffers, as many as tensor memory holds up to 16: the MMAs, and with them the stream of weights,
  // run on while the epilogue finishes a tile (4400 cycles) and meets the next one's scales (3500, from HBM)
  static constexpr int kCols = SHARE ? 128 * NMAT : 512;
  static constexpr int kDB = kCols / (NMAT * BN) < 16 ? kCols / (NMAT * BN) : 16;
  static constexpr int kTmemCols = kDB * NMAT * BN;    // a power of two, 256 or 512
  static constexpr int kBars = (2 * kStages + 2 * kDB + 3 + kSets + 1) / 2 * 2;   // even: what follows is 16-byte aligned
  static constexpr int kFixedBytes = 1024 + kStages * kStageBytes + kXBytes + kBars * 8 + kSets * 8 * BN * 4 + 64;
  static constexpr int smem_bytes(int E) { return kFixedBytes + 12 * (E + 1); }   // and the groups' table
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
  static_assert(smem_bytes(1024) <= 227 * 1024, "shared memory");
  // CTAs that `left` bytes of a SM's shared memory hold (1 KB of each is the system's)
  static constexpr int ctas_in(int left) { return left / (smem_bytes(1) + 1024); }
  static constexpr int kSmLeft = 228 * 1024 - smem_bytes(1) - 1024;   // beside one CTA
};
// Whatever CTAs of the SHARE kernels shared memory lets on a SM, calls on other streams among them, tensor memory has
// columns for: no CTA waits in the allocation, where the CTAs of two clusters could hold each other up without a limit.
// (The other stream kernels fill a SM's shared memory, the tile kernels its registers, which their split needs whole.)
template <int BN>
constexpr bool fp8_share_fits() {
  using GateUp = Fp8StreamCfg<2, BN, true>;
  using Down = Fp8StreamCfg<1, BN, true>;
  return GateUp::ctas_in(228 * 1024) == 1 && Down::ctas_in(228 * 1024) * Down::kTmemCols <= 512 &&
         GateUp::kTmemCols + Down::ctas_in(GateUp::kSmLeft) * Down::kTmemCols <= 512;
}
static_assert(fp8_share_fits<16>(), "tensor memory of the kernels that share a SM");


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

// barrier kinds of a wait timeout: the epilogue warps' own, the output staging's, the cluster's exchange
constexpr int kTagEpi = 9, kTagOut = 10, kTagX = 11;

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

__device__ __forceinline__ void fma2_to(unsigned long long& acc, uint32_t lo, uint32_t hi, unsigned long long s) {
  acc = fma2(pack2(__uint_as_float(lo), __uint_as_float(hi)), s, acc);
}

// The groups as tiles of BN rows, in shared memory: first[e] is expert e's
// first tile, first[E] their number.
struct Fp8Groups {
  int *first, *rb, *slot;
};
__device__ void fp8_group_table(const Fp8Params& p, int bn, const Fp8Groups& g, int* warp_sums) {
  const int per = (p.E + blockDim.x - 1) / blockDim.x, e0 = threadIdx.x * per;
  int sum = 0;
  for (int e = e0; e < min(p.E, e0 + per); ++e) {
    const int rb = __ldg(p.offsets + e);
    int n = __ldg(p.offsets + e + 1) - rb;
    const int slot = __ldg(p.slot_table + e);
    if (n > 0 && (slot < 0 || slot >= p.num_slots)) {
      if (blockIdx.x == 0) set_device_status(slot < 0 ? FT_DEV_NOT_RESIDENT : FT_DEV_BAD_INDEX);
      n = 0;
    }
    g.rb[e] = rb;
    g.slot[e] = slot;
    g.first[e] = sum;                    // within this thread's experts, for now
    sum += n > 0 ? (n + bn - 1) / bn : 0;
  }
  const int base = block_exclusive_scan(sum, warp_sums);
  for (int e = e0; e < min(p.E, e0 + per); ++e) g.first[e] += base;
  if (threadIdx.x == blockDim.x - 1) {
    g.first[p.E] = base + sum;
    g.rb[p.E] = __ldg(p.offsets + p.E);
  }
  __syncthreads();
}

// The walk of one CTA over its K blocks: tiles cid, cid + ncl, ..., of each the blocks [k0, k1).
struct Fp8Walk {
  const Fp8Params& p;
  const Fp8Groups& g;
  int bn, units, ncl, k0, k1;
  int u, kb;
  Fp8Unit d;
  __device__ Fp8Walk(const Fp8Params& p_, const Fp8Groups& g_, int bn_, int units_, int cid, int ncl_, int k0_, int k1_)
      : p(p_), g(g_), bn(bn_), units(units_), ncl(ncl_), k0(k0_), k1(k1_), u(cid), kb(k0_) { find(); }
  __device__ __forceinline__ bool more() const { return u < units; }
  __device__ __forceinline__ void find() {
    if (u >= units) return;
    const int tile = p.offsets ? u / p.feat_tiles : u % p.row_tiles;
    d.ft = p.offsets ? u - tile * p.feat_tiles : u / p.row_tiles;
    if (!p.offsets) {
      d.slot = 0;
      d.rb = tile * bn;
      d.nr = min(bn, p.rows - d.rb);
      return;
    }
    int lo = 0, hi = p.E;                // the last expert whose first tile is <= tile
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.first[mid] <= tile) lo = mid; else hi = mid;
    }
    const int t = tile - g.first[lo];
    d.slot = g.slot[lo];
    d.rb = g.rb[lo] + t * bn;
    d.nr = min(bn, g.rb[lo + 1] - d.rb);
  }
  __device__ __forceinline__ void next_tile() { u += ncl; kb = k0; find(); }
  __device__ __forceinline__ void next() { if (++kb == k1) next_tile(); }
};

// Abort::wait for what other CTAs of the cluster wrote.
__device__ __forceinline__ bool cluster_wait(const Abort& ab, uint64_t* bar, uint32_t parity, long long unit) {
  if (!ab.wait(bar, parity, kTagX, 0, unit)) return false;
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return true;
}

// The partial sums of a tile of nr rows (n < nr of acc[m][n]; this thread's
// weight row) to the CTAs that finish them, and back the sums of this CTA's
// columns: acc[m][j] becomes column rank * (BN / S) + j.
template <int NMAT, int BN, int S>
__device__ __forceinline__ bool fp8_exchange(float (&acc)[NMAT][BN], float* xbuf, uint64_t* x_full, uint64_t* x_free,
                                             uint32_t phase, int rank, int nr, int row, int lane, const Abort& ab,
                                             long long unit) {
  constexpr int C = BN / S;   // columns a CTA
  if (!__all_sync(0xFFFFFFFFu, cluster_wait(ab, x_free, phase ^ 1, unit))) return false;   // the last tile's are read
#pragma unroll
  for (int q = 0; q < S; ++q) {
    if (q * C >= nr) break;
    const uint32_t dst = cluster_addr(xbuf, q) + rank * (NMAT * C * 512) + row * 4;
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
      for (int j = 0; j < C; ++j)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + (m * C + j) * 512), "f"(acc[m][q * C + j]) : "memory");
  }
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  __syncwarp();
  if (lane < S)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(x_full, lane)) : "memory");
  if (!__all_sync(0xFFFFFFFFu, cluster_wait(ab, x_full, phase, unit))) return false;
  if (rank * C < nr) {
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
      for (int j = 0; j < C; ++j) {
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < S; ++q) sum += xbuf[((q * NMAT + m) * C + j) * 128 + row];
        acc[m][j] = sum;
      }
  }
  __syncwarp();
  if (lane < S)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(x_free, lane)) : "memory");
  return true;
}

// A tile is 128 weight rows x BN token rows.  The K blocks of one tile are
// shared by the `split` CTAs of a cluster, each of which streams its share
// of the weights (a full ring of them in flight a SM); the partial sums go
// through distributed shared memory: each CTA adds up, in the order of the
// CTAs (the same bits every time), and finishes BN / split of the columns.
// A tile's weights stand in memory longer than its token rows (`early`: the
// kernel before this one makes those rows): the first ring of weights is
// requested before that kernel has ended.
template <int NMAT, int BN, bool SHARE>
__global__ void __launch_bounds__(Fp8StreamCfg<NMAT, BN, SHARE>::kThreads, SHARE ? 2 : 1)
fp8_stream_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap tm_w0,
                  const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_rows) {
  using Cfg = Fp8StreamCfg<NMAT, BN, SHARE>;
  constexpr int NST = Cfg::kStages, DB = Cfg::kDB, DBS = DB / Cfg::kSets;   // DBS: accumulator buffers of one set
  extern __shared__ uint8_t smem_raw[];
  __shared__ int warp_sums[32];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* xbuf = reinterpret_cast<float*>(smem + NST * Cfg::kStageBytes);   // [source][matrix][BN / split][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NST * Cfg::kStageBytes + Cfg::kXBytes);
  uint64_t* empty = full + NST;
  uint64_t* d_full = empty + NST;
  uint64_t* d_empty = d_full + DB;
  uint64_t* drain_bar = d_empty + DB;
  uint64_t* x_full = drain_bar + 1;     // the cluster's partial sums of this CTA's columns are here
  uint64_t* x_free = x_full + 1;        // the cluster has read this CTA's partial sums
  uint64_t* epi_bar = x_free + 1;       // [set]
  // of each epilogue warp: a block's row scales [BN], and its maxima of h [BN]
  float* srow = reinterpret_cast<float*>(full + Cfg::kBars);
  uint32_t* tmax0 = reinterpret_cast<uint32_t*>(srow + Cfg::kSets * 4 * BN);
  uint32_t* tmem_slot = tmax0 + Cfg::kSets * 4 * BN;
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  Fp8Groups groups;
  groups.first = abort_flag + 1;
  groups.rb = groups.first + p.E + 1;
  groups.slot = groups.rb + p.E + 1;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp-uniform
  const int S = p.split;
  const int rank = S > 1 ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < DB; ++i) { mbar_init(&d_full[i], 1); mbar_init(&d_empty[i], 4); }
    mbar_init(drain_bar, 1);
    for (int i = 0; i < Cfg::kSets; ++i) mbar_init(&epi_bar[i], 4);
    mbar_init(x_full, 4 * S);
    mbar_init(x_free, 4 * S);
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(&tm_w0);
    if (NMAT > 1) prefetch_tmap(&tm_w1);
    prefetch_tmap(&tm_rows);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, Cfg::kTmemCols); tmem_relinquish(); }
  tc_fence_before();
  if (!p.early) pdl_wait();
  if (p.offsets) fp8_group_table(p, BN, groups, warp_sums);
  else __syncthreads();
  if (S > 1) cluster_arrive();   // this CTA's barriers are in place; the others' are waited for before their first use
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const Abort ab{abort_flag};
  const int nk = p.nk, per = (nk + S - 1) / S;
  const int units = p.offsets ? groups.first[p.E] * p.feat_tiles : p.row_tiles * p.feat_tiles;
  bool joined = false;   // whether this thread has waited for the cluster's CTAs
  Fp8Walk w(p, groups, BN, units, blockIdx.x / S, gridDim.x / S, rank * per, min(nk, (rank + 1) * per));

  if (warp == 0) {
    // ------------------------------------------------ TMA producer ---
    if (lane == 0) {
      uint32_t i = 0;
      auto weights = [&](const Fp8Walk& at, int s) {
        uint8_t* dst = smem + s * Cfg::kStageBytes;
        mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
        tma_load_3d(dst, &tm_w0, &full[s], at.kb * 128, at.d.ft * 128, at.d.slot);
        if (NMAT > 1) tma_load_3d(dst + kFp8WBytes, &tm_w1, &full[s], at.kb * 128, at.d.ft * 128, at.d.slot);
      };
      auto rows = [&](const Fp8Walk& at, int s) {
        tma_load_2d(smem + s * Cfg::kStageBytes + NMAT * kFp8WBytes, &tm_rows, &full[s], at.kb * 128, at.d.rb);
      };
      if (p.early) {
        Fp8Walk t = w;
        for (; i < NST && w.more(); ++i, w.next()) weights(w, i);
        pdl_wait();
        for (uint32_t j = 0; j < i; ++j, t.next()) rows(t, j);
      }
      for (; w.more(); ++i, w.next()) {
        const int s = i % NST;
        if (!ab.wait(&empty[s], ((i / NST) & 1) ^ 1, kTagWEmpty, i, w.u)) break;
        weights(w, s);
        rows(w, s);
      }
      for (uint32_t j = (i > NST ? i - NST : 0); j < i; ++j) {   // drain: every copy has landed
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&full[j % NST], (j / NST) & 1) && globaltimer_ns() - t0 < 1000000000ull) {}
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer ---
    uint32_t i = 0;
    uint32_t c = 0, other = 0;   // blocks given to the set at hand and to the other one
    uint32_t phase = 0;
    int s = 0, set = 0;
    bool ready = false;          // a test of a block's barriers takes some 85 cycles: made behind the block before it
    while (w.more()) {
      const uint32_t b = set * DBS + c % DBS;
      const uint32_t idesc = make_idesc_e4m3(128, (w.d.nr + 15) & ~15);
      if (!__all_sync(0xFFFFFFFFu, ready)) {
        const bool ok = ab.wait(&d_empty[b], ((c / DBS) & 1) ^ 1, kTagDEmpty, i, w.u) &&
                        ab.wait(&full[s], phase, kTagWFull, i, w.u);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
      }
      tc_fence_after();
      const int s1 = s + 1 == NST ? 0 : s + 1;
      const bool turn = Cfg::kSets == 2 && S == 1 && w.kb + 1 == w.k1;   // the next tile is the other set's
      const uint32_t c1 = turn ? other : c + 1;
      ready = mbar_test_wait(&d_empty[(turn ? set ^ 1 : set) * DBS + c1 % DBS], ((c1 / DBS) & 1) ^ 1);
      ready &= mbar_test_wait(&full[s1], s1 == 0 ? phase ^ 1 : phase);
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
      if (s1 == 0) phase ^= 1;
      s = s1;
      ++i;
      if (turn) {
        other = c + 1;
        set ^= 1;
      }
      c = c1;
      w.next();
    }
    if (i > 0) {   // drain: every MMA this warp issued has completed
      if (elect_one()) mma_commit(drain_bar);
      __syncwarp();
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < 1000000000ull) {}
    }
  } else {
    // ---------------------------------------------------- epilogue ---
    if (p.early) pdl_wait();
    pdl_launch_dependents();   // what follows fits beside this kernel only as its CTAs end
    const int quarter = warp & 3, set = (warp - 2) >> 2;
    // the sets take every kSets-th tile of this CTA; a split tile's exchange is one set's alone
    const int turns = S > 1 ? 1 : Cfg::kSets;
    const int row = quarter * 32 + lane;                 // weight row within the tile = tensor-memory lane
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    constexpr int kGroups = (BN + 31) / 32;
    EpiSync epi{epi_bar + set, ab, 0};
    float* sw = srow + (warp - 2) * BN;
    uint32_t* tmax = tmax0 + set * 4 * BN;
    uint32_t i = 0, x_phase = 0;                         // i: blocks of this set so far
    if (set > 0 && turns == 1) w.u = w.units;            // nothing for this set
    bool ok = true, ready = false;                       // ready: as of the MMA warp
    // Scales: lane j holds the weights' of block kb0 + j, 32 blocks at a time, and those of token row 32 q + j for
    // the next two blocks.  A tile's first ones are requested before the tile before it is finished.
    Fp8Unit d = {};
    const float* wp[NMAT];
    float wl[NMAT], sr[kGroups], sr1[kGroups], sr2[kGroups];
    auto row_scales = [&](int kb, float (&v)[kGroups]) {
#pragma unroll
      for (int q = 0; q < kGroups; ++q)
        v[q] = q * 32 + lane < d.nr && kb < w.k1 ? __ldg(p.sa + (d.rb + q * 32 + lane) * p.ld_sa + kb) : 0.0f;
    };
    auto weight_scales = [&](int kb) {
#pragma unroll
      for (int m = 0; m < NMAT; ++m) wl[m] = kb + lane < w.k1 ? __ldg(wp[m] + kb + lane) : 0.0f;
    };
    auto begin_tile = [&]() {
      d = w.d;
#pragma unroll
      for (int m = 0; m < NMAT; ++m) wp[m] = fp8_weight_scales(p, m, d.slot, d.ft);
      weight_scales(w.k0);
      row_scales(w.k0, sr1);
      row_scales(w.k0 + 1, sr2);
    };
    if (set > 0 && w.more()) w.next_tile();
    if (w.more()) begin_tile();
    for (; w.more() && ok; x_phase ^= 1) {
      const int n_eff = (d.nr + 15) & ~15;
      unsigned long long acc2[NMAT][BN / 2];
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int n = 0; n < BN / 2; ++n) acc2[m][n] = 0ull;
      for (int kb = w.k0; kb < w.k1; ++kb, ++i) {
        const int kj = (kb - w.k0) & 31;
        if (kj == 0 && kb > w.k0) weight_scales(kb);
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
          sr[q] = sr1[q];
          sr1[q] = sr2[q];
          if (BN >= 32 || lane < BN) sw[q * 32 + lane] = sr[q];
        }
        row_scales(kb + 2, sr2);
        __syncwarp();   // the row scales stand in shared memory
        const int b = set * DBS + i % DBS;
        if (!__all_sync(0xFFFFFFFFu, ready) &&
            !(ok = __all_sync(0xFFFFFFFFu, ab.wait(&d_full[b], (i / DBS) & 1, kTagDFull, i, w.u))))
          break;
        tc_fence_after();
        ready = mbar_test_wait(&d_full[set * DBS + (i + 1) % DBS], ((i + 1) / DBS) & 1);
        unsigned long long ws[NMAT];
#pragma unroll
        for (int m = 0; m < NMAT; ++m) {
          const float v = __shfl_sync(0xFFFFFFFFu, wl[m], kj);
          ws[m] = pack2(v, v);
        }
        const uint32_t dcol = tmem + lane_base + b * NMAT * BN;
#pragma unroll
        for (int c = 0; c < BN / 16; ++c) {
          if (c * 16 >= n_eff) break;
          uint32_t v[NMAT][16];
#pragma unroll
          for (int m = 0; m < NMAT; ++m) tmem_ld_32x32b_x16(dcol + m * BN + c * 16, v[m]);
          float4 s4[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) s4[n] = *reinterpret_cast<const float4*>(sw + c * 16 + 4 * n);
          tmem_wait_ld();
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const unsigned long long lo = pack2(s4[n].x, s4[n].y), hi = pack2(s4[n].z, s4[n].w);
#pragma unroll
            for (int m = 0; m < NMAT; ++m) {
              unsigned long long* a = &acc2[m][c * 8 + 2 * n];
              fma2_to(a[0], v[m][4 * n], v[m][4 * n + 1], mul2(lo, ws[m]));
              fma2_to(a[1], v[m][4 * n + 2], v[m][4 * n + 3], mul2(hi, ws[m]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[b]);
      }
      if (!ok) break;
      const Fp8Unit done = d;
      const long long u = w.u;
      w.next_tile();
      if (turns == 2) w.next_tile();
      if (w.more()) begin_tile();
      float acc[NMAT][BN];
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int n = 0; n < BN / 2; ++n) {
          const float2 f = unpack2(acc2[m][n]);
          acc[m][2 * n] = f.x;
          acc[m][2 * n + 1] = f.y;
        }
      if (Cfg::kXBytes > 0 && S > 1) {
        if (!joined) cluster_wait_all();
        joined = true;
        ok = S == 2   ? fp8_exchange<NMAT, BN, 2>(acc, xbuf, x_full, x_free, x_phase, rank, done.nr, row, lane, ab, u)
             : S == 4 ? fp8_exchange<NMAT, BN, 4>(acc, xbuf, x_full, x_free, x_phase, rank, done.nr, row, lane, ab, u)
                      : fp8_exchange<NMAT, BN, 8>(acc, xbuf, x_full, x_free, x_phase, rank, done.nr, row, lane, ab, u);
        if (!ok) break;
      }
      // this CTA's columns: token rows rb0 + j, j < nc
      const int c0 = rank * (BN / S), nc = min(done.nr - c0, BN / S);
      const long long rb0 = done.rb + c0;
      const int feat = done.ft * 128 + row;
      if constexpr (NMAT == 1) {
        if (feat < p.N) {
          const size_t at = rb0 * p.ldo + feat;
          if (p.out_type == FT_F32) {
#pragma unroll
            for (int j = 0; j < BN; ++j)
              if (j < nc) static_cast<float*>(p.out)[at + j * p.ldo] = acc[0][j];
          } else {
#pragma unroll
            for (int j = 0; j < BN; ++j)
              if (j < nc) static_cast<__nv_bfloat16*>(p.out)[at + j * p.ldo] = __float2bfloat16_rn(acc[0][j]);
          }
        }
      } else {
        // h = silu(gate) up; its scale is the maximum over the tile's 128 features (those past N are zeros)
#pragma unroll
        for (int j = 0; j < BN; ++j) {
          if (j >= nc) break;
          acc[0][j] = fp8_silu_mul(acc[0][j], acc[NMAT - 1][j]);
          const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, abs_bits(acc[0][j]));
          if (lane == 0) tmax[quarter * BN + j] = m;
        }
        if (!(ok = epi.sync(lane))) break;
        uint8_t* h = static_cast<uint8_t*>(p.out);
        const int hb = (p.N + kFp8Block - 1) / kFp8Block;
#pragma unroll
        for (int j = 0; j < BN; ++j) {
          if (j >= nc) break;
          const uint32_t m = max(max(tmax[j], tmax[BN + j]), max(tmax[2 * BN + j], tmax[3 * BN + j]));
          const Fp8Scale f = fp8_scale_of(__uint_as_float(m));
          if (feat < p.N) h[(rb0 + j) * p.ldo + feat] = uint8_t(fp8_codes2(acc[0][j], 0.0f, f));
          if (row == 0) p.hs[(rb0 + j) * hb + done.ft] = f.scale;
        }
        if (!(ok = epi.sync(lane))) break;   // the maxima are read before the next tile's are written
      }
    }
  }
  tc_fence_before();
  if (S > 1 && !joined) cluster_wait_all();
  __syncthreads();
  if (S > 1) cluster_sync();   // no CTA leaves while another may still write to it
  pdl_launch_dependents();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// --------------------------------------------------------- many rows ---

// PAIR: two CTAs of a cluster take one tile of 256 token rows (cta_group::2):
// each loads its own 128 rows and half of the 256 weight rows, so that a block
// costs 32 KB of shared-memory writes and reads a CTA where one CTA alone
// needs 48 KB of each for the same MMAs.
constexpr int kFp8OutChunk = 128 * 128;   // staged output: 128 rows of 128 bytes (64 bf16 or 32 fp32 features)

template <int NMAT, bool PAIR>
struct Fp8TileCfg {
  static constexpr int kRows = PAIR ? 256 : 128;                // token rows a tile
  // columns the epilogue reads at once
  static constexpr int kChunk = !PAIR && NMAT == 1 ? 16 : 32;
  static constexpr int kWRows = PAIR ? 128 : 256;               // weight rows this CTA loads
  static constexpr int kStages = PAIR || NMAT == 2 ? 4 : 3;
  static constexpr int kStageBytes = kFp8WBytes + kWRows * 128;
  static constexpr int kOutBytes = NMAT == 2 ? 2048 : 4 * kFp8OutChunk;   // gate/up: row maxima; else two chunks a half
  static constexpr int kBars = 2 * kStages + 2 * 4 + 2 + 4;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kOutBytes + kBars * 8 + 32;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};
constexpr int kFp8TileThreads = 384;   // warps for TMA, MMA, output stores and waiting; two epilogue warpgroups

// An arrive on a barrier of the pair.  It says only that this warp's tensor
// memory loads are done (they are waited for); a release at cluster scope
// would hold the warp until all its memory traffic is visible to the peer,
// some thousand cycles a block.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// The tensor-memory, TMA and MMA forms of one CTA or of a pair.  A pair's TMA
// loads (each CTA into its own shared memory, no multicast) complete on the
// leader's barrier; its commits arrive on both CTAs' barriers.
template <bool PAIR>
struct Fp8Pair {
  static __device__ __forceinline__ void alloc(uint32_t* dst) {
    if (PAIR) asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n"
                           " tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(dst)) : "memory");
    else { tmem_alloc(dst, 512); tmem_relinquish(); }
  }
  static __device__ __forceinline__ void dealloc(uint32_t tmem) {
    if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    else tmem_dealloc(tmem, 512);
  }
  static __device__ __forceinline__ void load_2d(void* dst, const void* map, uint32_t bar, int x, int y) {
    if (PAIR)
      asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                   " [%0], [%1, {%3, %4}], [%2];"
                   ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
    else
      asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                   " [%0], [%1, {%3, %4}], [%2];"
                   ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
  }
  static __device__ __forceinline__ void load_3d(void* dst, const void* map, uint32_t bar, int x, int y, int z) {
    if (PAIR)
      asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                   " [%0], [%1, {%3, %4, %5}], [%2];"
                   ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
    else
      asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                   " [%0], [%1, {%3, %4, %5}], [%2];"
                   ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
  }
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate) {
    if (PAIR)
      asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                   " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
                   ::"r"(d), "l"(a), "l"(b), "r"(make_idesc_e4m3(256, 128)), "r"(accumulate) : "memory");
    else
      mma_ss_f8(d, a, b, make_idesc_e4m3(128, 128), accumulate);
  }
  static __device__ __forceinline__ void commit(uint32_t bar) {
    if (PAIR)
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                   ::"r"(bar), "h"(uint16_t(3)) : "memory");
    else
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  }
};

// A box of shared memory (128-byte swizzled) to a 2-D tensor; one of the thread's bulk group.
__device__ __forceinline__ void tma_store_2d(const void* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
               ::"l"(map), "r"(smem_u32(src)), "r"(x), "r"(y) : "memory");
}

// Staged rows to an output without a tensor map, an element a lane.
__device__ __forceinline__ void fp8_store_rows(uint8_t* dst, long long pitch, const uint8_t* rows, int n, int nf, int esize,
                                            int lane) {
#pragma unroll 2
  for (int r = 0; r < n; ++r, dst += pitch) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int f = lane + 32 * q, byte = f * esize;   // of the row's 256 staged bytes
      if (f >= nf) continue;
      const uint8_t* src = rows + (byte >> 7) * kFp8OutChunk + r * 128 + ((((byte >> 4) & 7) ^ (r & 7)) << 4) + (byte & 15);
      if (esize == 4) reinterpret_cast<uint32_t*>(dst)[f] = *reinterpret_cast<const uint32_t*>(src);
      else reinterpret_cast<uint16_t*>(dst)[f] = *reinterpret_cast<const uint16_t*>(src);
    }
  }
}

// TMA_OUT: the output has a tensor map (a kernel without one has registers spilled by the plain stores).
template <int NMAT, bool PAIR, bool TMA_OUT>
__global__ void __launch_bounds__(kFp8TileThreads, 1)
fp8_tile_kernel(const Fp8Params p, const __grid_constant__ CUtensorMap tm_w0,
                const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_rows,
                const __grid_constant__ CUtensorMap tm_out) {
  using Cfg = Fp8TileCfg<NMAT, PAIR>;
  using Pair = Fp8Pair<PAIR>;
  constexpr int NST = Cfg::kStages, DB = 2;   // DB: accumulator buffers
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_stage = smem + NST * Cfg::kStageBytes;
  uint32_t* tmax = reinterpret_cast<uint32_t*>(out_stage);   // gate/up: [unit parity][half][128] row maxima
  uint64_t* full = reinterpret_cast<uint64_t*>(out_stage + Cfg::kOutBytes);
  uint64_t* empty = full + NST;
  uint64_t* d_full = empty + NST;         // [buffer][half]
  uint64_t* d_empty = d_full + 2 * DB;
  uint64_t* drain_bar = d_empty + 2 * DB;
  uint64_t* epi_bar = drain_bar + 1;
  uint64_t* out_full = epi_bar + 1;      // [half]
  uint64_t* out_empty = out_full + 2;    // [half]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(out_empty + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp-uniform
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2 * DB; ++i) { mbar_init(&d_full[i], 1); mbar_init(&d_empty[i], PAIR ? 8 : 4); }
    mbar_init(drain_bar, 1);
    mbar_init(epi_bar, 8);
    for (int i = 0; i < 2; ++i) { mbar_init(&out_full[i], 4); mbar_init(&out_empty[i], 1); }
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(&tm_w0);
    if (NMAT > 1) prefetch_tmap(&tm_w1);
    prefetch_tmap(&tm_rows);
  }
  if (warp == 1) Pair::alloc(tmem_slot);
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();   // the peer's barriers are in place
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const Abort ab{abort_flag};
  const int nk = p.nk;
  const int n_units = p.units ? *p.num_units : p.row_tiles * p.feat_tiles;
  const int u0 = PAIR ? blockIdx.x / 2 : blockIdx.x, du = PAIR ? gridDim.x / 2 : gridDim.x;

  // registers: 384 threads x 168 at launch = 128 x 56 + 256 x 224
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------------------------------------- TMA producer ---
      if (lane == 0) {
        uint32_t i = 0;
        bool ok = true;
        for (int u = u0; u < n_units && ok; u += du) {
          const Fp8Unit d = fp8_unit(p, u, Cfg::kRows);
          for (int kb = 0; kb < nk; ++kb, ++i) {
            const int s = i % NST;
            if (!(ok = ab.wait(&empty[s], ((i / NST) & 1) ^ 1, kTagWEmpty, i, u))) break;
            uint8_t* dst = smem + s * Cfg::kStageBytes;
            const uint32_t bar = PAIR ? cluster_addr(&full[s], 0) : smem_u32(&full[s]);
            if (rank == 0) mbar_arrive_expect_tx(&full[s], (PAIR ? 2 : 1) * Cfg::kStageBytes);
            Pair::load_2d(dst, &tm_rows, bar, kb * 128, d.rb + rank * 128);
            uint8_t* wdst = dst + kFp8WBytes;
            // Half h's 128 columns: NMAT 1 features 128 h .. of the tile's 256, NMAT 2 gate, then up of features
            // 64 h .. of its 128; of a pair's half, CTA 0 holds the first 64 columns' rows and CTA 1 the others'.
            if (NMAT == 2 && PAIR) {
              Pair::load_3d(wdst, rank ? &tm_w1 : &tm_w0, bar, kb * 128, d.ft * 128, d.slot);
            } else if (NMAT == 2) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                Pair::load_3d(wdst + h * kFp8WBytes, &tm_w0, bar, kb * 128, d.ft * 128 + h * 64, d.slot);
                Pair::load_3d(wdst + h * kFp8WBytes + kFp8WBytes / 2, &tm_w1, bar, kb * 128, d.ft * 128 + h * 64, d.slot);
              }
            } else if (PAIR) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                Pair::load_3d(wdst + h * kFp8WBytes / 2, &tm_w0, bar, kb * 128, d.ft * 256 + h * 128 + rank * 64, d.slot);
            } else {
              Pair::load_3d(wdst, &tm_w0, bar, kb * 128, d.ft * 256, d.slot);
            }
          }
        }
        // drain: the last copies have landed, as the MMAs that read them are done
        for (uint32_t j = (i > NST ? i - NST : 0); j < i; ++j) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(&empty[j % NST], (j / NST) & 1) && globaltimer_ns() - t0 < 1000000000ull) {}
        }
      }
    } else if (warp == 1 && rank == 0) {
      // ----------------------------------------------- MMA issuer ---
      // Each K block as two 128-column halves with accumulators of their own, so
      // that half 0 is read back while half 1 is multiplied: the round trip of
      // a buffer (MMAs, commit, the epilogue's wake-up and reads, its arrive)
      // is some 1200 cycles against the 1024 of two blocks' MMAs; as one
      // 256-column buffer a block it was 1500, and that set the pace.
      // Warp 3 does the waiting, half by half and one half ahead, and the two
      // meet at a named barrier: an mbarrier test takes some 85 cycles to
      // answer, and with two of them a half this warp's own instructions were
      // the bound (900 cycles a block).  Where warp 3 has given up, it only
      // passes: the MMAs then work on what is there, and the status is set.
      const uint64_t rd0 = make_sdesc_sw128(smem_u32(smem)), wd0 = make_sdesc_sw128(smem_u32(smem + kFp8WBytes));
      const uint32_t d_bar = smem_u32(d_full), e_bar = smem_u32(empty);
      int s = 0, b = 0;
      bool issued = false;
      for (int u = u0; u < n_units; u += du) {
        for (int kb = 0; kb < nk; ++kb) {
          const uint64_t rd = rd0 + s * (Cfg::kStageBytes >> 4), wd = wd0 + s * (Cfg::kStageBytes >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            named_bar_sync(kBarHandoff, 64);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                Pair::mma(tmem + b * 256 + h * 128, rd + 2 * j, wd + h * (Cfg::kWRows * 128 / 2 >> 4) + 2 * j, j > 0);
              Pair::commit(d_bar + 8 * (2 * b + h));
              if (h == 1) Pair::commit(e_bar + 8 * s);
            }
            __syncwarp();
          }
          issued = true;
          if (++s == NST) s = 0;
          b ^= 1;
        }
      }
      if (issued) {   // drain
        if (elect_one()) Pair::commit(smem_u32(drain_bar));
        __syncwarp();
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < 1000000000ull) {}
      }
    } else if (warp == 3 && rank == 0) {
      // ------------------------------------------- the MMAs' waits ---
      uint32_t i = 0;
      int s = 0, phase = 0;
      bool ok = true;
      for (int u = u0; u < n_units; u += du) {
        for (int kb = 0; kb < nk; ++kb, ++i) {
          const uint32_t b = i & 1, dp = ((i >> 1) & 1) ^ 1;
          ok = ok && ab.wait(&full[s], phase, kTagWFull, i, u);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && ab.wait(&d_empty[2 * b + h], dp, kTagDEmpty, i, u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            named_bar_sync(kBarHandoff, 64);
          }
          if (++s == NST) { s = 0; phase ^= 1; }
        }
      }
    } else if (warp == 2 && NMAT == 1 && TMA_OUT) {
      // -------------------------------------------- output stores ---
      // The staged features of each half (128 bf16; or 64 fp32, twice), as
      // 32-row boxes of 128 bytes, behind the next tile's sums: stores from the
      // epilogue warps themselves held them, and with them the MMAs, for a
      // quarter of the time.  The rows of a box that would reach past the
      // group's go by 16-byte stores.
      const bool f32 = p.out_type == FT_F32;
      const int esize = f32 ? 4 : 2, per = 128 / esize;   // features a chunk
      uint32_t n = 0;
      bool ok = true;
      for (int u = u0; u < n_units && ok; u += du) {
        const Fp8Unit d = fp8_unit(p, u, Cfg::kRows);
        const int rb = d.rb + rank * 128, nr = max(0, min(d.nr - int(rank) * 128, 128)), boxes = nr / 32;
        for (int pass = 0; pass < (f32 ? 2 : 1) && ok; ++pass, ++n) {
          for (int half = 0; half < 2; ++half) {
            if (!(ok = __all_sync(0xFFFFFFFFu, ab.wait(&out_full[half], n & 1, kTagOut, n, u)))) break;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              const uint8_t* stage = out_stage + (half * 2 + c) * kFp8OutChunk;
              const int f0 = d.ft * 256 + half * 128 + (2 * pass + c) * per, nf = min(per, p.N - f0);
              if (nf <= 0) break;
              if (lane < boxes) tma_store_2d(&tm_out, stage + lane * 32 * 128, f0, rb + lane * 32);
#pragma unroll 1
              for (int row = boxes * 32 + (lane >> 3); row < nr; row += 4) {
                const int piece = lane & 7, f = piece * (16 / esize);
                const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 128 + ((piece ^ (row & 7)) << 4));
                uint8_t* dst = static_cast<uint8_t*>(p.out) + ((rb + row) * p.ldo + f0 + f) * esize;
                if (f < nf) *reinterpret_cast<uint4*>(dst) = x;   // N ends on a piece
              }
            }
            asm volatile("cp.async.bulk.commit_group;\n cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&out_empty[half]);
          }
        }
      }
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // -------------------------------------------------- epilogue ---
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;                 // token row within the CTA's 128 = tensor-memory lane
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    uint32_t d_empty_addr[DB];
#pragma unroll
    for (int b = 0; b < DB; ++b) d_empty_addr[b] = PAIR ? cluster_addr(&d_empty[2 * b + half], 0) : 0;
    EpiSync epi{epi_bar, ab, 0};
    uint32_t i = 0, staged = 0;
    bool ok = true;
    int parity = 0;
    constexpr int kCh = Cfg::kChunk, kNc = 128 / kCh;
    // A tile's descriptor and its first two blocks' scales are fetched behind
    // the tile before it: two dependent round trips to memory.
    Fp8Unit d = {};
    const float *sr, *sw0, *sw1;
    float a, w0, w1, an, w0n, w1n;
    const int last = nk - 1;
    auto fetch_scales = [&]() {
      sr = p.sa + (long long)(int(rank) * 128 + row < d.nr ? d.rb + int(rank) * 128 + row : d.rb) * p.ld_sa;
      // a feature block past the end has no scales: its columns are zeros, and block 0's scale does
      const int block = NMAT == 2 ? d.ft : d.ft * 2 + half;
      sw0 = fp8_weight_scales(p, 0, d.slot, block * kFp8Block < p.N ? block : 0);
      sw1 = NMAT == 2 ? fp8_weight_scales(p, 1, d.slot, block) : sw0;
      const int k1 = min(1, last);
      a = __ldg(sr);
      w0 = __ldg(sw0);
      w1 = NMAT == 2 ? __ldg(sw1) : 0.0f;
      an = __ldg(sr + k1);
      w0n = __ldg(sw0 + k1);
      w1n = NMAT == 2 ? __ldg(sw1 + k1) : 0.0f;
    };
    if (u0 < n_units) {
      d = fp8_unit(p, u0, Cfg::kRows);
      fetch_scales();
    }
    for (int u = u0; u < n_units && ok; u += du, parity ^= 1) {
      const int rb = d.rb + rank * 128, nr_here = d.nr - int(rank) * 128;
      const bool live = row < nr_here;
      unsigned long long acc[64];   // NMAT 1: 128 columns; NMAT 2: gate of 64 features, then up
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0ull;
      // Chunks of kCh columns in two register buffers, the next chunk's load in
      // flight behind one chunk's sums -- also across blocks: the last chunk's
      // sums stand behind the next block's first load.
      uint32_t v[2][kCh];
      if (!(ok = __all_sync(0xFFFFFFFFu, ab.wait(&d_full[2 * (i & 1) + half], (i >> 1) & 1, kTagDFull, i, u)))) break;
      tc_fence_after();
      const uint32_t dcol = tmem + lane_base + half * 128;
      tmem_ld_cols(dcol + (i & 1) * 256, v[0]);
      for (int kb = 0; kb < nk; ++kb, ++i) {
        const uint32_t b = i & 1;
        const float s0 = a * w0, s1 = a * w1;
        const unsigned long long p0 = pack2(s0, s0);
        const unsigned long long p1 = NMAT == 2 ? pack2(s1, s1) : p0;
        a = an;
        w0 = w0n;
        w1 = w1n;
        const int k2 = min(kb + 2, last);
        an = __ldg(sr + k2);
        w0n = __ldg(sw0 + k2);
        if (NMAT == 2) w1n = __ldg(sw1 + k2);
        bool ready = false;
        auto sums = [&](int c) {
#pragma unroll
          for (int n = 0; n < kCh / 2; ++n)
            fma2_to(acc[c * (kCh / 2) + n], v[c & 1][2 * n], v[c & 1][2 * n + 1], c < kNc / 2 ? p0 : p1);
        };
#pragma unroll
        for (int c = 0; c < kNc - 1; ++c) {
          tmem_wait_ld();
          tmem_ld_cols(dcol + b * 256 + (c + 1) * kCh, v[(c + 1) & 1]);
          if (c == kNc - 2) ready = mbar_test_wait(&d_full[2 * (b ^ 1) + half], ((i + 1) >> 1) & 1);
          sums(c);
        }
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster(b ? d_empty_addr[1] : d_empty_addr[0]);
          else mbar_arrive(&d_empty[2 * b + half]);
        }
        if (kb == last) {
          sums(kNc - 1);
        } else {
          if (!ready) {
            sums(kNc - 1);
            if (!(ok = __all_sync(0xFFFFFFFFu, ab.wait(&d_full[2 * (b ^ 1) + half], ((i + 1) >> 1) & 1, kTagDFull, i + 1, u))))
              break;
          }
          tc_fence_after();
          tmem_ld_cols(dcol + (b ^ 1) * 256, v[0]);
          if (ready) sums(kNc - 1);
        }
      }
      if (!ok) break;
      const int ft = d.ft;
      if (u + du < n_units) d = fp8_unit(p, u + du, Cfg::kRows);
      if constexpr (NMAT == 1) {
        // each thread its row's features, to the store warp: 16-byte piece q of a row at q ^ (row % 8)
        uint8_t* stage = out_stage + half * 2 * kFp8OutChunk + row * 128;
        const bool f32 = p.out_type == FT_F32;
        auto give = [&](auto pass_tag) {   // the accumulators' indices have to be constants
          constexpr int pass = decltype(pass_tag)::value;
          if constexpr (TMA_OUT) {
            if (!(ok = __all_sync(0xFFFFFFFFu, ab.wait(&out_empty[half], (staged & 1) ^ 1, kTagOut, staged, u)))) return;
            ++staged;
          }
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            uint32_t o[4];
            if (f32) {
              const float2 x = unpack2(acc[pass * 32 + 2 * q]), y = unpack2(acc[pass * 32 + 2 * q + 1]);
              o[0] = __float_as_uint(x.x); o[1] = __float_as_uint(x.y);
              o[2] = __float_as_uint(y.x); o[3] = __float_as_uint(y.y);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 x = unpack2(acc[4 * q + e]);
                const __nv_bfloat162 t = __floats2bfloat162_rn(x.x, x.y);
                o[e] = *reinterpret_cast<const uint32_t*>(&t);
              }
            }
            *reinterpret_cast<uint4*>(stage + (q >> 3) * kFp8OutChunk + (((q & 7) ^ (row & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
          if constexpr (TMA_OUT) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&out_full[half]);
          } else {
            __syncwarp();
            const int esize = f32 ? 4 : 2, f0 = ft * 256 + half * 128 + pass * 64;
            fp8_store_rows(static_cast<uint8_t*>(p.out) + ((long long)(rb + quarter * 32) * p.ldo + f0) * esize,
                           p.ldo * esize, out_stage + half * 2 * kFp8OutChunk + quarter * 32 * 128,
                           min(32, nr_here - quarter * 32), min(256 / esize, p.N - f0), esize, lane);
            __syncwarp();
          }
        };
        give(std::integral_constant<int, 0>());
        if (f32 && ok) give(std::integral_constant<int, 1>());
        fetch_scales();
        if (!ok) break;
      } else {
        // h of this thread's 64 features; its scale is the maximum over the row's 128 (those past N are zeros)
        float h[64], hm = 0.0f;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 g = unpack2(acc[c]), up = unpack2(acc[32 + c]);
          h[2 * c] = fp8_silu_mul(g.x, up.x);
          h[2 * c + 1] = fp8_silu_mul(g.y, up.y);
          hm = fmaxf(hm, fmaxf(fabsf(h[2 * c]), fabsf(h[2 * c + 1])));   // leaves NaN out
        }
        uint32_t m = __float_as_uint(hm);
        tmax[parity * 256 + half * 128 + row] = m;
        fetch_scales();
        if (!(ok = epi.sync(lane))) break;
        m = max(m, tmax[parity * 256 + (half ^ 1) * 128 + row]);
        const Fp8Scale f = fp8_scale_of(__uint_as_float(m));
        const int f0 = ft * 128 + half * 64;
        if (live) {
          if (half == 0) p.hs[(long long)(rb + row) * ((p.N + kFp8Block - 1) / kFp8Block) + ft] = f.scale;
          if (f0 < p.N) {   // N is a multiple of 64
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (rb + row) * p.ldo + f0);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t o[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                o[q] = fp8_codes4(h[16 * c + 4 * q], h[16 * c + 4 * q + 1], h[16 * c + 4 * q + 2], h[16 * c + 4 * q + 3], f);
              dst[c] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();   // neither CTA leaves while the other may still signal it
  pdl_launch_dependents();
  if (warp == 1) {
    tc_fence_after();
    Pair::dealloc(tmem);
  }
}

// ------------------------------------------------------ prep kernels ---

// One launch: blocks [0, sched.nsched) build the two work lists and clear the
// counters (prep_schedule of ffn.cu), the others write the token rows in FP8
// in permuted order, eight lanes a group of 128 values.
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
  const int H = p.sched.H;
  const uint32_t nb = (H + kFp8Block - 1) / kFp8Block, groups = uint32_t(p.sched.P) * nb;   // < 2^31
  const uint32_t block = blockIdx.x - p.sched.nsched, stride = (gridDim.x - p.sched.nsched) * 32u;
  const int sub = threadIdx.x & 7;
  Raw16<__nv_bfloat16> raw;
  uint32_t r = 0, b = 0;
  auto fetch = [&](uint32_t g) {
    r = g / nb;
    b = g - r * nb;
    const bool live = g < groups;
    const int src = live ? __ldg(p.sched.perm_src + r) : -1, t = src / p.sched.k_top;
    const bool known = src >= 0 && t < p.T;
    if (live && !known && b == 0 && sub == 0) set_device_status(FT_DEV_BAD_INDEX);
    const int k0 = b * kFp8Block + sub * 16;   // H is a multiple of 64: all sixteen or none
    if (known && k0 < H) raw.load(p.x + (long long)t * H + k0);
    else raw.zero();
  };
  uint32_t g = (block * 256u + threadIdx.x) >> 3;
  fetch(g);
  for (uint32_t w = (block * 256u + (threadIdx.x & ~31u)) >> 3; w < groups; w += stride) {
    float v[16];
    raw.to(v);
    const uint32_t row = r, c = b;
    const bool live = g < groups;
    g += stride;
    if (w + stride < groups) fetch(g);
    const Fp8Scale f = fp8_scale_of(group_max(v));
    if (!live) continue;
    if (sub == 0) p.scales[(long long)row * nb + c] = f.scale;
    const int k0 = c * kFp8Block + sub * 16;
    if (k0 < H) *reinterpret_cast<uint4*>(p.codes + (long long)row * H + k0) = fp8_codes16(v, f);
  }
}

// The rows of x, already quantised once a token, to their places in expert
// order: a warp a row.  Bound by the writes of k copies.  The kernel above does
// a token's arithmetic k times instead: at 4096 tokens x 2048, k = 8, the FFN
// takes 295 us with it and 282 with these two launches (1500 tokens x 2880,
// k = 4: the same within the noise).
struct Fp8SpreadParams {
  PrepParams sched;
  int T;
  const uint8_t* from_codes;   // [T, H]
  const float* from_scales;    // [T, ceil(H/128)]
  uint8_t* codes;              // [P, H]
  float* scales;
};
__global__ void __launch_bounds__(256) fp8_spread_kernel(const Fp8SpreadParams p) {
  pdl_enter();
  if (int(blockIdx.x) < p.sched.nsched) {
    prep_schedule(p.sched, blockIdx.x);
    return;
  }
  const int lane = threadIdx.x & 31, H = p.sched.H, nb = (H + kFp8Block - 1) / kFp8Block;
  const int stride = (gridDim.x - p.sched.nsched) * 8;
  for (int r = (blockIdx.x - p.sched.nsched) * 8 + (threadIdx.x >> 5); r < p.sched.P; r += stride) {
    const int src = __ldg(p.sched.perm_src + r), t = src / p.sched.k_top;
    const bool known = src >= 0 && t < p.T;
    if (!known && lane == 0) set_device_status(FT_DEV_BAD_INDEX);
    const uint4* from = reinterpret_cast<const uint4*>(p.from_codes + (long long)t * H);   // H is a multiple of 64
    uint4* to = reinterpret_cast<uint4*>(p.codes + (long long)r * H);
#pragma unroll 4
    for (int c = lane; c < H / 16; c += 32) to[c] = known ? __ldg(from + c) : make_uint4(0u, 0u, 0u, 0u);
    for (int c = lane; c < nb; c += 32)
      p.scales[(long long)r * nb + c] = known ? __ldg(p.from_scales + (long long)t * nb + c) : 0.0f;
  }
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

// The output [rows, N] as boxes of 32 rows x 128 bytes; false where its pitch
// or address does not allow a map, or a row does not end on 16 bytes (a store
// cuts its box there: with N = 333 fp32 columns it wrote zeros to 333 .. 335).
static bool make_fp8_out_map(void* out, int out_type, long long rows, int N, long long ldo, CUtensorMap* m) {
  auto enc = tensor_map_encoder();
  const int esize = out_type == FT_F32 ? 4 : 2;
  if (!enc || (ldo * esize) % 16 || (N * esize) % 16 || (reinterpret_cast<uintptr_t>(out) & 15)) return false;
  const cuuint64_t dims[2] = {cuuint64_t(N), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ldo * esize)};
  const cuuint32_t box[2] = {cuuint32_t(128 / esize), 32};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, out_type == FT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch in clusters of `cluster` CTAs, allowed to begin while the kernel before it ends.
template <typename... KArgs, typename... Args>
static cudaError_t launch_fp8_grid(void (*kern)(KArgs...), int grid, int threads, int smem, int cluster, cudaStream_t s,
                                   Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// CTAs that the device can hold at once in clusters of `cluster`, of one kernel
// at one CTA a SM (a property of the device, kept per kernel and device).
template <typename K>
static int fp8_cluster_ctas(K kern, int threads, int smem, int cluster, int num_sms, std::atomic<int>* kept) {
  if (cluster == 1) return num_sms;
  int n = kept->load();
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms / cluster * cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1) clusters = num_sms / cluster;
    n = std::min(clusters, num_sms / cluster) * cluster;
    kept->store(n);
  }
  return n;
}

// units: the tiles as far as the host can tell, most: their bound.
//
// The K blocks of a tile are shared by the split (1, 2, 4, 8) with the least
// time on the busiest cluster, counted in K blocks: tiles a cluster takes x
// blocks a CTA, three more a split tile for its exchange (some 2.5 us against
// 0.75 us a block of gate/up).
template <int NMAT, int BN, bool SHARE>
static cudaError_t launch_fp8_stream(Fp8Params p, double units, long long most, int num_sms, const CUtensorMap& w0,
                                     const CUtensorMap& w1, const CUtensorMap& rows, cudaStream_t s) {
  using Cfg = Fp8StreamCfg<NMAT, BN, SHARE>;
  static std::atomic<int> allowed[64], ctas[64][4];   // by device
  auto kern = fp8_stream_kernel<NMAT, BN, SHARE>;
  constexpr int kMost = Cfg::smem_bytes(1024);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  dev &= 63;
  if (!allowed[dev].load()) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e == cudaSuccess && SHARE)
      e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    allowed[dev].store(1);
  }
  int cap = num_sms;
  double best = ceil(units / num_sms) * p.nk;
  p.split = 1;
  for (int i = 1; Cfg::kXBytes > 0 && i < 4 && (1 << i) <= p.nk; ++i) {
    const int S = 1 << i, per = (p.nk + S - 1) / S;
    if ((S - 1) * per >= p.nk) continue;   // a CTA without a block
    const int n = fp8_cluster_ctas(kern, Cfg::kThreads, kMost, S, num_sms, &ctas[dev][i]);
    const double cost = ceil(units / (n / S)) * (per + 3);
    if (cost < best - 1e-9) { best = cost; p.split = S; cap = n; }
  }
  const int grid = int(std::min<long long>(most * p.split, cap));
  return launch_fp8_grid(kern, grid, Cfg::kThreads, Cfg::smem_bytes(p.E), p.split, s, p, w0, w1, rows);
}
static int fp8_tile_grid(long long units, bool pair, int num_sms) {
  return pair ? 2 * int(std::min<long long>(units, num_sms / 2)) : int(std::min<long long>(units, num_sms));
}
template <int NMAT, bool PAIR, bool TMA_OUT>
static cudaError_t launch_fp8_tile(const Fp8Params& p, long long units, int num_sms, const CUtensorMap& w0,
                                   const CUtensorMap& w1, const CUtensorMap& rows, const CUtensorMap& out, cudaStream_t s) {
  static std::atomic<uint64_t> done[64];
  auto kern = fp8_tile_kernel<NMAT, PAIR, TMA_OUT>;
  constexpr int kSmem = Fp8TileCfg<NMAT, PAIR>::kSmemBytes;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!done[dev & 63].load()) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    done[dev & 63].store(1);
  }
  return launch_fp8_grid(kern, fp8_tile_grid(units, PAIR, num_sms), kFp8TileThreads, kSmem, PAIR ? 2 : 1, s, p, w0, w1,
                         rows, out);
}
// units: the tiles as far as the host can tell, most: their bound.
template <int NMAT>
static cudaError_t launch_fp8_any(int bn, Fp8Params p, long long out_rows, double units, long long most,
                                  const CUtensorMap& w0, const CUtensorMap& w1, const CUtensorMap& rows, cudaStream_t s) {
  const int num_sms = device_sm_count();
  CUtensorMap out = rows;
  const bool mapped = bn < 128 || NMAT == 2 || make_fp8_out_map(p.out, p.out_type, out_rows, p.N, p.ldo, &out);
  switch (bn) {
    case 16:
      return p.share ? launch_fp8_stream<NMAT, 16, true>(p, units, most, num_sms, w0, w1, rows, s)
                     : launch_fp8_stream<NMAT, 16, false>(p, units, most, num_sms, w0, w1, rows, s);
    case 32: return launch_fp8_stream<NMAT, 32, false>(p, units, most, num_sms, w0, w1, rows, s);
    case 64: return launch_fp8_stream<NMAT, 64, false>(p, units, most, num_sms, w0, w1, rows, s);
    case 128:   // experts: H is a multiple of 64, every output has a map
      return mapped ? launch_fp8_tile<NMAT, false, true>(p, most, num_sms, w0, w1, rows, out, s) : cudaErrorInvalidValue;
    default:
      if constexpr (NMAT == 1)
        if (!mapped) return launch_fp8_tile<NMAT, true, false>(p, most, num_sms, w0, w1, rows, out, s);
      return launch_fp8_tile<NMAT, true, true>(p, most, num_sms, w0, w1, rows, out, s);
  }
}

// Rows, padded to tiles of b, of a group of `mean` rows that spread by their square root.
static double fp8_padded(double mean, int b) {
  double sum = 0.0;
  for (double q : {-1.4, -0.7, -0.3, 0.0, 0.3, 0.7, 1.4}) sum += b * ceil(std::max(1.0, mean + q * sqrt(mean)) / b) / 7;
  return sum;
}
// Token rows a tile takes (16, 32, 64: the stream kernel; 128, 256: the tile
// kernel on one CTA or a pair).  For few rows a quarter more than the mean, so
// that most groups of an even spread are one tile.  A pair takes some 0.9 of the
// time for the same padded rows, but pads more.  The FFN in pairs and in tiles
// of 128: groups of some 187 rows, 32 of them 2880 x 2880 253 and 275 us, 128 of
// them 2048 x 768 216 and 225 to 250; 2048 rows 38 and 40; 250 rows 313 and 311;
// 256 rows 300 and 270; 125 rows 245 and 214; 75 rows 240 and 169; 4096 skewed
// tokens of 128 groups 324 and 281.
static int fp8_rows_tile(double mean) {
  const double rows = 1.25 * mean;
  if (rows <= 64) return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  return 0.9 * fp8_padded(mean, 256) < fp8_padded(mean, 128) ? 256 : 128;
}
// Rows of a token box, and of a weight box of `nmat` matrices.
static int fp8_row_box(int bn) { return std::min(bn, 128); }
static int fp8_weight_box(int bn, int nmat) {
  return bn < 128 ? 128 : bn == 128 ? (nmat == 2 ? 64 : 256) : (nmat == 2 ? 128 : 64);
}

struct Fp8GemmPlan {
  int bn, row_tiles, feat_tiles;
};
// The stream kernel while one tile takes all rows, or while its tiles are no
// more than the SMs (65 x 1024 x 2048: 7.6 us against 10.5 of the tile kernel,
// 200 x 2048 x 2048: 9.9 against 11.0); past that its CTAs take a second tile
// (128 x 8192 x 2048: 15.9 us against 11.5, 64 x 16384 x 2048: 15.9 against
// 11.4) and each reads the weights again.
static Fp8GemmPlan plan_fp8_gemm(int M, int N, int num_sms) {
  Fp8GemmPlan pl{};
  const long long jobs = ((M + 31LL) / 32) * ((N + 127LL) / 128);
  pl.bn = M <= 16 ? 16 : (M <= 32 || jobs <= num_sms) ? 32 : 256;
  pl.row_tiles = (M + pl.bn - 1) / pl.bn;
  pl.feat_tiles = pl.bn >= 128 ? (N + 255) / 256 : (N + 127) / 128;
  return pl;
}

static cudaError_t launch_fp8_gemm(const uint8_t* a, long long lda, const float* sa, long long ld_sa, const uint8_t* b,
                                   long long ldb, const float* sb, long long ld_sb, int M, int N, int K, void* out,
                                   int out_type, long long ldo, cudaStream_t s, const char** why) {
  const int num_sms = device_sm_count();
  const Fp8GemmPlan pl = plan_fp8_gemm(M, N, num_sms);
  CUtensorMap tm_a, tm_b;
  if (!make_fp8_map(a, M, K, lda, 1, 16, fp8_row_box(pl.bn), false, &tm_a) ||
      !make_fp8_map(b, N, K, ldb, 1, ldb * N, fp8_weight_box(pl.bn, 1), true, &tm_b)) {
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
  const long long units = (long long)pl.row_tiles * pl.feat_tiles;
  ProfileScope prof(FT_KERNEL_FP8_GEMM, s);
  return launch_fp8_any<1>(pl.bn, p, M, double(units), units, tm_b, tm_b, tm_a, s);
}

struct Fp8FfnPlan {
  int bn, mt1, mt2;                 // token rows a tile takes; feature tiles of gate/up and down
  double tiles;                     // token tiles, as far as the host can tell
  long long max_units1, max_units2;
  bool spread;                      // quantise by token, then copy to the rows
  size_t off_x, off_xs, off_h, off_hs, off_t, off_ts, off_units1, off_units2, off_counts, total;
};
static Fp8FfnPlan plan_fp8_ffn(int T, int H, int I, int E, int k) {
  Fp8FfnPlan p{};
  const long long P = (long long)T * k;
  const double distinct = std::max(1.0, E * (1.0 - pow(1.0 - double(k) / E, double(T))));
  p.bn = fp8_rows_tile(double(P) / distinct);
  p.mt1 = fp8_blocks(I);
  p.mt2 = p.bn >= 128 ? (H + 255) / 256 : fp8_blocks(H);
  const long long tiles = std::min<long long>(E, P) + P / p.bn;
  p.max_units1 = tiles * p.mt1;
  p.max_units2 = tiles * p.mt2;
  const bool stream = p.bn < 128;
  p.tiles = ceil(distinct) * std::max(1.0, ceil(double(P) / distinct / p.bn));
  size_t o = 0;
  p.off_x = o;      o = align256(o + size_t(P) * H);
  p.off_xs = o;     o = align256(o + size_t(P) * fp8_blocks(H) * 4);
  p.off_h = o;      o = align256(o + size_t(P) * I);
  p.off_hs = o;     o = align256(o + size_t(P) * fp8_blocks(I) * 4);
  p.spread = !stream && k > 1;
  p.off_t = o;      o = align256(o + (p.spread ? size_t(T) * H : 0));
  p.off_ts = o;     o = align256(o + (p.spread ? size_t(T) * fp8_blocks(H) * 4 : 0));
  p.off_units1 = o; o = align256(o + (stream ? 0 : size_t(p.max_units1) * 16));
  p.off_units2 = o; o = align256(o + (stream ? 0 : size_t(p.max_units2) * 16));
  p.off_counts = o; o = align256(o + 16);
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
  bool ok = make_fp8_map(w + pl.off_x, P, H, H, 1, 16, fp8_row_box(pl.bn), false, &tm_x) &&
            make_fp8_map(w + pl.off_h, P, I, I, 1, 16, fp8_row_box(pl.bn), false, &tm_h);
  for (int m = 0; m < 3; ++m)
    ok = ok && make_fp8_map(pool + L.codes_off[m], rows[m], Ks[m], Ks[m], L.num_slots, L.slot_bytes,
                            fp8_weight_box(pl.bn, m == FT_DOWN ? 1 : 2), true, &tm[m]);
  if (!ok) {
    *why = "ft_moe_ffn_fp8: cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  int4* units1 = reinterpret_cast<int4*>(w + pl.off_units1);
  int4* units2 = reinterpret_cast<int4*>(w + pl.off_units2);
  int* counts = reinterpret_cast<int*>(w + pl.off_counts);
  cudaError_t e;
  PrepParams sp{};
  sp.offsets = offsets;
  sp.slot_table = slot_table;
  sp.E = E;
  sp.num_slots = L.num_slots;
  // The stream kernel finds its tiles itself.  Else a block a unit a thread (4096 skewed tokens of 128 experts, FFN: 282
  // us, in one block 284).
  sp.nsched = stream ? 0 : int(std::min<long long>(32, std::max<long long>(1, (pl.max_units1 + pl.max_units2) / 256)));
  sp.bn1 = sp.bn2 = pl.bn;
  sp.mt1 = pl.mt1;
  sp.mt2 = pl.mt2;
  sp.s1 = sp.s2 = 1;
  sp.units1 = units1;
  sp.units2 = units2;
  sp.counts = counts;
  sp.perm_src = perm_src;
  sp.P = P;
  sp.k_top = k;
  sp.H = H;
  if (pl.spread) {
    Fp8SpreadParams pp{};
    pp.sched = sp;
    pp.T = T;
    pp.from_codes = w + pl.off_t;
    pp.from_scales = reinterpret_cast<const float*>(w + pl.off_ts);
    pp.codes = w + pl.off_x;
    pp.scales = reinterpret_cast<float*>(w + pl.off_xs);
    e = launch_fp8_quant(x, FT_BF16, T, H, H, w + pl.off_t, H, reinterpret_cast<float*>(w + pl.off_ts), fp8_blocks(H), s);
    if (e != cudaSuccess) return e;
    const int ctas = std::min((P + 7) / 8, device_sm_count() * 8);
    ProfileScope prof(FT_KERNEL_PREP, s);
    e = launch_pdl(fp8_spread_kernel, dim3(sp.nsched + ctas), dim3(256), 0, s, pp);
  } else {
    Fp8PrepParams pp{};
    pp.sched = sp;
    pp.x = static_cast<const __nv_bfloat16*>(x);
    pp.T = T;
    pp.codes = w + pl.off_x;
    pp.scales = reinterpret_cast<float*>(w + pl.off_xs);
    const long long groups = (long long)P * fp8_blocks(H);
    ProfileScope prof(FT_KERNEL_PREP, s);
    e = launch_pdl(fp8_prep_kernel, dim3(sp.nsched + fp8_quant_grid(groups, device_sm_count())), dim3(256), 0, s, pp);
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
  if (stream) {
    // Before this kernel stands the prep kernel, which writes neither weights nor groups, and which began
    // its own work, and so let this one begin, only when all before it had ended.
    p.offsets = offsets;
    p.slot_table = slot_table;
    p.E = E;
    p.num_slots = L.num_slots;
    p.early = 1;
    // While gate/up has a tile a SM at most (128 experts, 2048 x 768, k = 8: one token 17.1 us, apart 20.2; three 28.9
    // and 32.0); with more, the shorter rings cost more than the early weights give (16 tokens 82.8 and 79.6 us, 64
    // tokens 118.2 and 111.4).
    p.share = pl.bn == 16 && pl.tiles * pl.mt1 <= device_sm_count();
  } else {
    p.units = units1;
    p.num_units = counts;
  }
  p.feat_tiles = pl.mt1;
  p.out = w + pl.off_h;
  p.ldo = I;
  p.hs = reinterpret_cast<float*>(w + pl.off_hs);
  {
    ProfileScope prof(FT_KERNEL_FP8_GATE_UP, s);
    e = launch_fp8_any<2>(pl.bn, p, P, pl.tiles * pl.mt1, pl.max_units1, tm[FT_GATE], tm[FT_UP], tm_x, s);
  }
  if (e != cudaSuccess) return e;
  p.sa = reinterpret_cast<const float*>(w + pl.off_hs);
  p.ld_sa = fp8_blocks(I);
  p.sb[0] = p.sb[1] = reinterpret_cast<const float*>(pool + L.scales_off[FT_DOWN]);
  p.ld_sb = L.ld_scale[FT_DOWN] / 4;
  p.nk = fp8_blocks(I);
  p.N = H;
  if (!stream) {
    p.units = units2;
    p.num_units = counts + 1;
  }
  p.feat_tiles = pl.mt2;
  p.out = out;
  p.out_type = out_type;
  p.ldo = H;
  ProfileScope prof(FT_KERNEL_FP8_DOWN, s);
  return launch_fp8_any<1>(pl.bn, p, P, pl.tiles * pl.mt2, pl.max_units2, tm[FT_DOWN], tm[FT_DOWN], tm_h, s);
}

}  // namespace ftmoe
