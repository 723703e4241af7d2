// Products whose rows are grouped by expert, in bf16 and in block-scaled e4m3, on
// tcgen05 (a dense 8-bit linear is the case of one group).
//
//   Fwd  Y_e  = X_e W_e^T        Dx  dX_e = dY_e W_e        Dw  dW_e = dY_e^T X_e
//
// with X_e the rows [offsets[e], offsets[e + 1]) of X. In e4m3 every 128 values of a
// row share a scale and every 128 x 128 block of W shares one, so with k running
// over blocks of 128
//
//   Y[m, n] = sum_k sa[m, k] sb[n / 128, k] (sum_{j in block k} qa[m, j] qb[n, j]).
//
// The inner sums run on the tensor cores, 128 values deep, into a fresh TMEM buffer
// for each k; the outer sum is one fp32 multiply-add per value in the registers of
// the epilogue warps, which read buffer k while the tensor cores fill buffer k + 1.
// In bf16 the tensor cores sum over all of K and the epilogue reads once per tile (Dw, which
// stays in fp32: every 256 rows).
//
// One persistent CTA per SM, or one CTA pair per two SMs (cta_group::2, tiles of 256 x
// 256: each CTA stages its 128 rows of A and its 128 columns of B, so a byte from L2
// feeds twice the products that it does in a 128 x 128 tile). Roles:
//   warp 0      TMA producer
//   warp 1      TMEM allocation, MMA issue (even CTA of a pair)
//   warps 2, 3  e4m3: products of the scales to shared memory, four steps at a time;
//               Dw: ends of groups
//   warps 4..   epilogue, 4 lane quadrants x column groups: each warp owns 32 rows x 128
//               columns (64 in 128-column tiles), in registers
// In 256-column tiles an epilogue thread holds 128 sums and 64 values in flight; the first
// warpgroup gives up registers for that (168 x 384 = 56 x 128 + 224 x 256). 16 epilogue
// warps of 64 columns have 96 registers at most and spill: the e4m3 forward at 8192 x 11008
// x 4096 took 567 us with them and takes 376.
// Stage: 128 rows (or columns) x 128 bytes of K for each operand, 128-byte swizzle,
// K-major as stored along K, MN-major where the reduction runs over rows.
//
// Groups end where they end: A rows past a group's last row are loaded (or left as
// they were in shared memory) and multiplied, and never stored; products of rows are
// independent, so they cannot reach a stored one. B's tensor map has the expert as its
// third dimension, so columns of A past K meet zeros and not the next expert's rows.
// In Dw the rows are summed over, so the last step of a group is cleared in shared
// memory past the group's last row in both operands (a zero in one only would let a
// NaN of another expert's row through).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "expert_gemm.cuh"
#include "gemm.cuh"
#include "internal.cuh"
#include "nf4_device.cuh"
#include "ptx.cuh"

namespace qlb {

namespace {

struct ExpertParams {
  int M, E;
  int n_cols;            // columns of D
  int tiles_n;           // ceil(n_cols / BN)
  int tiles_r;           // Dw: row tiles of D per expert
  int nk;                // K steps (Fwd, Dx)
  int split, k_part;     // SPLIT: CTAs a tile, K steps of each (a multiple of 4)
  int d_rows;            // Dw: rows of D per expert
  int a_box;             // rows of A per TMA box: 128, or 32 where groups are small
  const int32_t* offsets;
  const float* sa;
  const float* sb;
  int nb_a;              // scales per row of A
  int sa_vec;            // rows of scales start on 16 bytes
  int nb_n;              // column blocks of sb (clamps the ragged last tile)
  int64_t sb_e, sb_n, sb_k;   // strides of sb: expert, column block, K block
  uint16_t* d;
  int64_t ld_d;
  int* status;
};

template <bool PAIR_, int BN_, bool F8_, ExpertMode MODE_, bool SPLIT_ = false>
struct ExpertCfg {
  static constexpr bool PAIR = PAIR_, F8 = F8_, WIDE = BN_ == 256;
  static constexpr bool SPLIT = SPLIT_;                 // K over a cluster of 2, 4 or 8 CTAs
  static_assert(WIDE || (BN_ == 128 && !PAIR), "tile widths");
  static_assert(!SPLIT || (!WIDE && MODE_ != ExpertMode::Dw), "K is split in 128 x 128 tiles");
  static constexpr ExpertMode MODE = MODE_;
  static constexpr bool DW = MODE == ExpertMode::Dw;
  static constexpr bool A_MN = DW, B_MN = MODE != ExpertMode::Fwd;
  static constexpr int BM = PAIR ? 256 : 128, BN = BN_;
  static constexpr int BCTA = PAIR ? 128 : BN;          // columns of B that a CTA stages
  static constexpr int kElem = F8 ? 1 : 2;
  static constexpr int BK = 128 / kElem;                // K per step: 128 bytes
  static constexpr int kChunk = 128 / kElem;            // MN-major: columns in 128 bytes
  static constexpr int kA = 128 * 128, kB = BCTA * 128;  // bytes per CTA and stage
  static constexpr int kStage = kA + kB;
  static constexpr int STAGES = !PAIR && WIDE ? 3 : 5;
  static constexpr int kCols = WIDE ? 128 : 64;         // columns per epilogue warp
  static constexpr int kEpiWarps = 4 * (BN / kCols);
  static constexpr int kThreads = (4 + kEpiWarps) * 32;
  static constexpr int kRoleRegs = 56, kEpiRegs = 224;  // WIDE
  static_assert(!WIDE || (kThreads == 384 && kRoleRegs * 128 + kEpiRegs * 256 <= 168 * 384), "register split");
  // Steps that the tensor cores sum in TMEM before the epilogue adds them to its registers: one
  // scale block in e4m3; all of K where D is rounded to bf16; four, 256 rows, in Dw, whose
  // fp32 result would show more (the tensor cores' adder cuts off where an fp32 addition
  // rounds, so the error grows with the additions in a row: over 16384 rows 1.9e-5 of dW's
  // norm summed in one go, 2.7e-7 so, 3.7e-7 by an fp32 product; 191 against 198 us at 8192
  // rows, 4096 x 4096).
  static constexpr int kSum = F8 ? 1 : DW ? 4 : 1 << 30;
  static constexpr int kBufs = F8 ? 512 / BN : 2;       // TMEM buffers of BN columns
  static constexpr int kTmemCols = kBufs * BN;
  static constexpr int kPassCols = DW ? 32 : 64;        // D columns in 128 bytes
  static constexpr int kStgBufs = 1;               // staging buffers per epilogue warp
  static constexpr int kStaging = kEpiWarps * kStgBufs * 4096;   // 32 rows x 128 bytes each
  static constexpr int kBlocksN = BN / 128;
  static constexpr int kScaleSlots = 3;
  static constexpr int kScaleSlot = 4 * kBlocksN * 512; // 4 steps x column blocks x 128 rows
  static constexpr int kScaleOff = STAGES * kStage + kStaging;
  static constexpr int kBarOff = kScaleOff + (F8 ? kScaleSlots * kScaleSlot : 0);
  static constexpr int kNumBars = 3 * STAGES + 2 * kBufs + 1 + 2 * kScaleSlots;
  static constexpr int kTableOff = kBarOff + kNumBars * 8 + 16;
  static constexpr int kSmem = kTableOff + 2 * (kMaxExperts + 1) * 4 + 1024;
  static_assert(kSmem <= 232448, "shared memory budget");
  // SPLIT: one warp's sums, 32 lanes x kCols fp32, from one of the other CTAs.
  static constexpr int kPart = 32 * kCols * 4;
  static_assert(!SPLIT || kEpiWarps * kPart <= STAGES * kStage, "room for the parts");
};

// acc += v * s for two values at once.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t s2) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s2));
}
__device__ __forceinline__ uint64_t dup2(float s) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(s));
  return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t a, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(a));
}

struct ExpertTile {
  int e, n0, nk;
  int kb0;            // SPLIT: this CTA's first step (0 otherwise); nk counts from it
  int row0, rows;     // Fwd, Dx: first row of the tile in A and D, rows of the group from there
                      // Dw: first row of D in the expert, rows of D from there
  int k_row0, k_rows; // Dw: the group's rows
};

// Within an expert tiles run in bands of kBand row tiles, over a band's rows first and then
// the columns, so that the tiles in flight cover a near-square patch of D and share both
// operands. `e` only moves up.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_in_band(int r, int mt, int tiles_n, int& m, int& n) {
  const int band = r / (kBand * tiles_n);
  const int h = min(kBand, mt - band * kBand);
  r -= band * kBand * tiles_n;
  n = r / h;
  m = band * kBand + r - n * h;
}
template <class C>
__device__ __forceinline__ ExpertTile expert_tile(const ExpertParams& p, const int* starts, const int* tiles, int t,
                                                  int& e) {
  ExpertTile x;
  x.kb0 = 0;
  if constexpr (C::DW) {
    const int per = p.tiles_r * p.tiles_n;
    e = t / per;
    int m, n;
    tile_in_band(t - e * per, p.tiles_r, p.tiles_n, m, n);
    x.row0 = m * C::BM;
    x.rows = p.d_rows - x.row0;
    x.n0 = n * C::BN;
    x.k_row0 = starts[e];
    x.k_rows = starts[e + 1] - starts[e];
    x.nk = (x.k_rows + C::BK - 1) / C::BK;
  } else {
    const int v = t / p.tiles_n;
    while (tiles[e + 1] <= v) ++e;
    int m, n;
    tile_in_band(t - tiles[e] * p.tiles_n, tiles[e + 1] - tiles[e], p.tiles_n, m, n);
    x.row0 = starts[e] + m * C::BM;
    x.rows = starts[e + 1] - x.row0;
    x.n0 = n * C::BN;
    x.nk = p.nk;
    if constexpr (C::SPLIT) {
      x.kb0 = min(p.nk, int(cluster_ctarank()) * p.k_part);
      x.nk = min(p.k_part, p.nk - x.kb0);
    }
    x.k_row0 = x.k_rows = 0;
  }
  x.e = e;
  return x;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmD, const ExpertParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(smem);
  const uint32_t bars = base + C::kBarOff;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (C::STAGES + s); };
  auto tfull_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + b); };
  auto tempty_bar = [&](int b) { return bars + 8u * (2 * C::STAGES + C::kBufs + b); };
  constexpr int kB0 = 2 * C::STAGES + 2 * C::kBufs;
  auto tail_bar = [&](int i) { return bars + 8u * (kB0 + i); };
  auto sfull_bar = [&](int s) { return bars + 8u * (kB0 + C::STAGES + s); };
  auto sempty_bar = [&](int s) { return bars + 8u * (kB0 + C::STAGES + C::kScaleSlots + s); };
  const uint32_t drain_bar = bars + 8u * (kB0 + C::STAGES + 2 * C::kScaleSlots);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 8 * C::kNumBars);
  int* starts = reinterpret_cast<int*>(smem + C::kTableOff);
  int* tiles = starts + kMaxExperts + 1;

  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = C::PAIR ? cluster_ctarank() : 0u;
  // (SPLIT: as many clusters as tiles, so each loop over tiles below runs at most once.)
  const int unit = C::PAIR ? int(blockIdx.x >> 1) : C::SPLIT ? int(blockIdx.x) / p.split : int(blockIdx.x);
  const int units = C::PAIR ? int(gridDim.x >> 1) : C::SPLIT ? int(gridDim.x) / p.split : int(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), C::PAIR ? 2 : 1);   // one arrival per CTA's producer
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), (C::PAIR ? 2 : 1) * C::kEpiWarps);
    }
    if constexpr (C::F8) {
      for (int s = 0; s < C::kScaleSlots; ++s) {
        mbar_init(sfull_bar(s), 64);
        mbar_init(sempty_bar(s), C::kEpiWarps);
      }
    }
    for (int s = 0; s < C::STAGES; ++s) mbar_init(tail_bar(s), 1);
    mbar_init(drain_bar, 1);
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    if constexpr (C::PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), C::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
      tmem_relinquish();
    }
  }
  pdl_wait();
  pdl_launch();
  // Group table: starts[e] is the running maximum of the offsets clamped to [0, M] (so
  // whatever they hold, groups lie inside A and do not overlap), tiles[e] the row tiles
  // of the groups before e.
  if (warp == 0) {
    if (p.offsets == nullptr) {
      if (lane == 0) {
        starts[0] = 0;
        starts[1] = p.M;
        tiles[0] = 0;
        tiles[1] = (p.M + C::BM - 1) / C::BM;
      }
    } else {
      int run = 0, sum = 0, prev = 0;
      bool bad = false;
      for (int i0 = 0; i0 <= p.E; i0 += 32) {
        const int i = i0 + int(lane);
        const int raw = i <= p.E ? ld_global(p.offsets + i) : 0;
        const int c = min(max(raw, 0), p.M);
        int v = max(c, run);
        for (int d = 1; d < 32; d <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, d);
          if (int(lane) >= d) v = max(v, u);
        }
        if (i <= p.E && (raw != c || v != c)) bad = true;
        int before = __shfl_up_sync(0xffffffffu, v, 1);
        if (lane == 0) before = prev;
        // row tiles of group i - 1, which ends at v
        int n = (i >= 1 && i <= p.E) ? (v - before + C::BM - 1) / C::BM : 0;
        for (int d = 1; d < 32; d <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, n, d);
          if (int(lane) >= d) n += u;
        }
        if (i <= p.E) {
          starts[i] = v;
          tiles[i] = sum + n;
        }
        run = prev = __shfl_sync(0xffffffffu, v, 31);
        sum += __shfl_sync(0xffffffffu, n, 31);
      }
      if (__any_sync(0xffffffffu, bad) && lane == 0) set_status_site(p.status, QLORA_ERR_SHAPE, 60);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (C::PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int num_tiles = C::DW ? p.E * p.tiles_r * p.tiles_n : tiles[p.E] * p.tiles_n;
  constexpr uint64_t kDrainNs = 100000000ull;

  if (warp < 4) {
  if constexpr (C::WIDE) regs_down<C::kRoleRegs>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
      uint32_t s = 0, ph = 1, ntail = 0;   // stage, and the parity that says it is free
      uint32_t issued = 0;
      int e = 0;
      bool ok = true;
      for (int t = unit; t < num_tiles && ok; t += units) {
        const ExpertTile x = expert_tile<C>(p, starts, tiles, t, e);
        const int a_rows = min(128, max(0, x.rows - int(rank) * 128));
        const int boxes = C::A_MN || C::PAIR ? 1 : (a_rows + p.a_box - 1) / p.a_box;
        const int b0 = x.n0 + int(rank) * C::BCTA;    // this CTA's columns of B
        const int a0 = x.row0 + int(rank) * 128;      // this CTA's rows of D
        for (int kb = 0; kb < x.nk; ++kb) {
          if (!mbar_wait_lazy(empty_bar(s), ph)) {
            set_status_site(p.status, QLORA_ERR_TIMEOUT, 61);
            ok = false;
            break;
          }
          const uint32_t a_s = base + s * C::kStage, b_s = a_s + C::kA;
          const bool tail = C::DW && x.k_rows - kb * C::BK < C::BK;
          uint32_t bar;
          if (tail) {
            // landed on a barrier of its own, which warp 2 waits on; it hands the stage over
            bar = tail_bar(ntail % C::STAGES);
            ++ntail;
            mbar_arrive_expect_tx(bar, C::kStage);
          } else if constexpr (C::PAIR) {
            // The even CTA's barrier counts both CTAs' bytes.
            bar = mapa_shared(full_bar(s), 0);
            if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * C::kStage);
            else mbar_arrive_remote(bar);
          } else {
            bar = full_bar(s);
            mbar_arrive_expect_tx(bar, (C::A_MN ? C::kA : boxes * p.a_box * 128) + C::kB);
          }
          const int k0 = (x.kb0 + kb) * C::BK;
          auto load2 = [&](uint32_t dst, const CUtensorMap* m, int cx, int cy) {
            if (C::PAIR && !tail) tma_load_2d_pair(dst, m, bar, cx, cy);
            else tma_load_2d(dst, m, bar, cx, cy);
          };
          auto load3 = [&](uint32_t dst, const CUtensorMap* m, int cx, int cy) {
            if (C::PAIR && !tail) tma_load_3d_pair(dst, m, bar, cx, cy, x.e);
            else tma_load_3d(dst, m, bar, cx, cy, x.e);
          };
          if constexpr (C::DW) {
#pragma unroll
            for (int c = 0; c < 2; ++c) load2(a_s + c * 8192, &tmA, a0 + 64 * c, x.k_row0 + k0);
#pragma unroll
            for (int c = 0; c < C::BCTA / 64; ++c) load2(b_s + c * 8192, &tmB, b0 + 64 * c, x.k_row0 + k0);
          } else {
            for (int b = 0; b < boxes; ++b) load2(a_s + b * p.a_box * 128, &tmA, k0, a0 + b * p.a_box);
            if constexpr (!C::B_MN) {
#pragma unroll
              for (int c = 0; c < C::BCTA / 128; ++c) load3(b_s + c * 16384, &tmB, k0, b0 + c * 128);
            } else {
#pragma unroll
              for (int c = 0; c < C::BCTA / C::kChunk; ++c)
                load3(b_s + c * C::BK * 128, &tmB, b0 + c * C::kChunk, k0);
            }
          }
          ++issued;
          if (++s == C::STAGES) { s = 0; ph ^= 1u; }
        }
      }
      // Do not leave while copies may still be landing (after an error; else all are consumed).
      if (!ok && rank == 0) {
        for (uint32_t k = 0; k < uint32_t(C::STAGES) && k < issued; ++k) {
          const uint32_t i2 = issued - 1 - k;
          mbar_wait(full_bar(i2 % C::STAGES), (i2 / C::STAGES) & 1u, kDrainNs);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc = C::F8 ? make_idesc_e4m3(C::BM, C::BN, C::A_MN, C::B_MN)
                                       : make_idesc_bf16(C::BM, C::BN, C::A_MN, C::B_MN);
      // K advance per instruction (32 bytes of K): inside a K-major row, or that many
      // 128-byte rows of an MN-major tile.
      constexpr uint32_t mn_adv = (32u / C::kElem) * 128u;
      constexpr uint32_t a_adv = C::A_MN ? mn_adv : 32u, b_adv = C::B_MN ? mn_adv : 32u;
      constexpr uint32_t mn_lbo = C::BK * 128u;   // bytes between MN-major column chunks
      constexpr uint32_t a_lbo = C::A_MN ? mn_lbo : 16u, b_lbo = C::B_MN ? mn_lbo : 16u;
      const uint64_t ad0 = make_smem_desc(base, a_lbo, 1024u, kSwizzle128B);
      const uint64_t bd0 = make_smem_desc(base + C::kA, b_lbo, 1024u, kSwizzle128B);
      uint32_t s = 0, ph = 0, u = 0;
      int e = 0;
      bool ok = true;
      for (int t = unit; t < num_tiles && ok; t += units) {
        const ExpertTile x = expert_tile<C>(p, starts, tiles, t, e);
        for (int kb = 0; kb < x.nk; ++kb) {
          const uint32_t buf = u % C::kBufs;
          if (kb % C::kSum == 0) {
            if (!mbar_wait_lazy(tempty_bar(buf), ((u / C::kBufs) & 1u) ^ 1u)) {
              set_status_site(p.status, QLORA_ERR_TIMEOUT, 63);
              ok = false;
              break;
            }
          }
          // (cluster scope where the other CTA's generic stores, a cleared tail, are handed over)
          const bool tail = C::PAIR && C::DW && x.k_rows - kb * C::BK < C::BK;
          if (!(tail ? mbar_wait_cluster(full_bar(s), ph) : mbar_wait_lazy(full_bar(s), ph))) {
            set_status_site(p.status, QLORA_ERR_TIMEOUT, 64);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = ad0 + uint64_t(s * (C::kStage >> 4)), bd = bd0 + uint64_t(s * (C::kStage >> 4));
          const uint32_t d = tmem + buf * C::BN;
#pragma unroll
          for (uint32_t kk = 0; kk < 4; ++kk) {
            const uint64_t a2 = ad + uint64_t((kk * a_adv) >> 4), b2 = bd + uint64_t((kk * b_adv) >> 4);
            const uint32_t acc = (kk > 0 || kb % C::kSum > 0) ? 1u : 0u;
            if constexpr (C::PAIR) {
              if constexpr (C::F8) tc_mma_f8_pair(d, a2, b2, idesc, acc);
              else tc_mma_bf16_pair(d, a2, b2, idesc, acc);
            } else {
              if constexpr (C::F8) tc_mma_f8(d, a2, b2, idesc, acc);
              else tc_mma_bf16(d, a2, b2, idesc, acc);
            }
          }
          if constexpr (C::PAIR) tc_commit_pair_mc(empty_bar(s), 3);
          else tc_commit(empty_bar(s));
          if (kb % C::kSum == C::kSum - 1 || kb == x.nk - 1) {
            if constexpr (C::PAIR) tc_commit_pair_mc(tfull_bar(buf), 3);
            else tc_commit(tfull_bar(buf));
            ++u;
          }
          if (++s == C::STAGES) { s = 0; ph ^= 1u; }
        }
      }
      // All MMAs of this thread are complete once drain_bar flips.
      if constexpr (C::PAIR) tc_commit_pair_mc(drain_bar, 1);
      else tc_commit(drain_bar);
      mbar_wait_lazy(drain_bar, 0, kDrainNs);
    }
  } else if (C::DW && warp == 2) {
    // ------------------------------------------------------------ ends of groups
    // Clears the last step of a group past its last row in both operands. (In the producer
    // the wait for the step's copies held up the next tile's: every group has such a step,
    // and with 256 rows a group it is one in five.)
    uint32_t it = 0, ntail = 0;
    int e = 0;
    for (int t = unit; t < num_tiles; t += units) {
      const ExpertTile x = expert_tile<C>(p, starts, tiles, t, e);
      it += x.nk;
      const int valid = x.k_rows - (x.nk - 1) * C::BK;
      if (x.nk == 0 || valid == C::BK) continue;
      // (a whole tile's steps may pass before: 4 us for each are ten times what they take)
      const uint64_t limit = 2000000000ull + 4000ull * uint64_t(x.nk);
      if (!__all_sync(0xffffffffu, mbar_wait_lazy(tail_bar(ntail % C::STAGES), (ntail / C::STAGES) & 1u, limit))) {
        if (lane == 0) set_status_site(p.status, QLORA_ERR_TIMEOUT, 62);
        break;
      }
      ++ntail;
      const int s = (it - 1) % C::STAGES;
      const uint4 z = make_uint4(0, 0, 0, 0);
      for (int c = 0; c < C::kStage / 8192; ++c) {
        uint8_t* chunk = smem + s * C::kStage + c * 8192;
        for (int i = valid * 8 + int(lane); i < 512; i += 32) reinterpret_cast<uint4*>(chunk)[i] = z;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if constexpr (C::PAIR) mbar_arrive_cluster(mapa_shared(full_bar(s), 0));
        else mbar_arrive(full_bar(s));
      }
    }
  } else {
    // ------------------------------------------------------------ scales
    // The products sa sb of the tile's 128 rows and column blocks, four steps at a time, two
    // rows a thread. Rows past the group's end take its last row's scales (in bounds; their
    // products are not stored), steps past the last one take its.
    if constexpr (C::F8) {
      const int t0 = int(threadIdx.x) - 64;
      uint32_t g = 0;
      int e = 0;
      bool ok = true;
      for (int t = unit; t < num_tiles && ok; t += units) {
        const ExpertTile x = expert_tile<C>(p, starts, tiles, t, e);
        const int r0 = int(rank) * 128 + t0;
        const float* ra = p.sa + int64_t(x.row0 + min(r0, x.rows - 1)) * p.nb_a + x.kb0;
        const float* rb = p.sa + int64_t(x.row0 + min(r0 + 64, x.rows - 1)) * p.nb_a + x.kb0;
        const float* sb = p.sb + x.e * p.sb_e + x.kb0 * p.sb_k;
        for (int k0 = 0; k0 < x.nk; k0 += 4, ++g) {
          const int s = g % C::kScaleSlots;
          float a[2][4], w[C::kBlocksN][4];
          if (p.sa_vec) {
            const float4 u = ld_global(reinterpret_cast<const float4*>(ra + k0));
            const float4 v = ld_global(reinterpret_cast<const float4*>(rb + k0));
            a[0][0] = u.x; a[0][1] = u.y; a[0][2] = u.z; a[0][3] = u.w;
            a[1][0] = v.x; a[1][1] = v.y; a[1][2] = v.z; a[1][3] = v.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              a[0][j] = ld_global(ra + min(k0 + j, x.nk - 1));
              a[1][j] = ld_global(rb + min(k0 + j, x.nk - 1));
            }
          }
#pragma unroll
          for (int b = 0; b < C::kBlocksN; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[b][j] = ld_global(sb + min((x.n0 >> 7) + b, p.nb_n - 1) * p.sb_n + min(k0 + j, x.nk - 1) * p.sb_k);
          if (!__all_sync(0xffffffffu, mbar_wait_lazy(sempty_bar(s), ((g / C::kScaleSlots) & 1u) ^ 1u))) {
            if (lane == 0) set_status_site(p.status, QLORA_ERR_TIMEOUT, 66);
            ok = false;
            break;
          }
          float* dst = reinterpret_cast<float*>(smem + C::kScaleOff + s * C::kScaleSlot) + t0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int b = 0; b < C::kBlocksN; ++b)
#pragma unroll
              for (int h = 0; h < 2; ++h) dst[(j * C::kBlocksN + b) * 128 + 64 * h] = a[h][j] * w[b][j];
          mbar_arrive(sfull_bar(s));
        }
      }
    }
  }
  if constexpr (C::SPLIT) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  } else {
    // ------------------------------------------------------------ epilogue
    if constexpr (C::WIDE) regs_up<C::kEpiRegs>();
    const uint32_t q = warp & 3u;                 // TMEM lane quadrant this warp may read
    const int cg = int(warp - 4) >> 2;            // column group
    const uint32_t stg0 = base + C::STAGES * C::kStage + (warp - 4) * (C::kStgBufs * 4096u);
    const uint32_t trow = tmem + ((q * 32u) << 16) + cg * C::kCols;
    uint32_t npass = 0;
    uint32_t u = 0, g = 0;
    int e = 0;
    bool ok = true;
    for (int t = unit; t < num_tiles && ok; t += units) {
      const ExpertTile x = expert_tile<C>(p, starts, tiles, t, e);
      const int first = int(rank) * 128 + int(q) * 32;       // this warp's first row in the tile
      const int rows = min(32, x.rows - first);              // rows to store (may be <= 0)
      const int col0 = x.n0 + cg * C::kCols;
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = 0;
      // Adds s times the next TMEM buffer to acc, and hands the buffer back.
      auto take = [&](float s) {
        const uint32_t buf = u % C::kBufs;
        if (!__all_sync(0xffffffffu, mbar_wait_lazy(tfull_bar(buf), (u / C::kBufs) & 1u))) {
          if (lane == 0) set_status_site(p.status, QLORA_ERR_TIMEOUT, 65);
          ok = false;   // (and on, so that the sums have one path: they are not stored)
        }
        ++u;
        tc_fence_after();
        const uint64_t s2 = dup2(s);
        constexpr int kLoads = C::kCols / 64;
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
          uint64_t v[32];
          tmem_ld_wait_32x32b_x64_pairs(trow + buf * C::BN + c * 64, v);
          if (c + 1 == kLoads) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if constexpr (C::PAIR) mbar_arrive_remote(mapa_shared(tempty_bar(buf), 0));
                else mbar_arrive(tempty_bar(buf));
              }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) fma2(acc[c * 32 + i], v[i], s2);
        }
      };
      if constexpr (C::F8) {
        for (int k = 0; k < x.nk && ok; k += 4, ++g) {
          const uint32_t slot = g % C::kScaleSlots;
          if (!__all_sync(0xffffffffu, mbar_wait_lazy(sfull_bar(slot), (g / C::kScaleSlots) & 1u))) {
            if (lane == 0) set_status_site(p.status, QLORA_ERR_TIMEOUT, 67);
            ok = false;
          }
          const uint32_t f = base + C::kScaleOff + slot * C::kScaleSlot +
                             ((cg * C::kCols / 128) * 128 + q * 32 + lane) * 4;
          const int n = min(4, x.nk - k);
          // Four in a row without a loop between them where the registers last: at 2048 rows,
          // 4096 x 4096, 40.5 us in 128 x 128 tiles against 48.5 (53 with the tests of each step in
          // the loop); 256-column tiles would spill (61 us against 40). (With K split 24 bytes a thread spill.)
          if (!C::WIDE && n == 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) take(lds_f32(f + j * C::kBlocksN * 512));
          } else {
#pragma unroll 1
            for (int j = 0; j < n; ++j) take(lds_f32(f + j * C::kBlocksN * 512));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sempty_bar(slot));
        }
      } else {
        for (int k = 0; k < x.nk && ok; k += C::kSum) take(1.f);
      }
      if constexpr (C::SPLIT) {
        // Each CTA finishes the warps w = its rank (mod the cluster's CTAs): the others send it
        // those warps' sums, into its ring, which is idle once every CTA is past its products,
        // and it adds them to its own in the order of their ranks.
        const int krank = int(cluster_ctarank()), w = int(warp) - 4;
        const int owner = w % p.split, per = C::kEpiWarps / p.split;
        auto slot = [&](int from) { return base + uint32_t(from * per + w / p.split) * C::kPart + lane * 16u; };
        cluster_sync();
        if (owner != krank && rows > 0) {
          const uint32_t dst = mapa_shared(slot(krank - (krank > owner)), owner);
#pragma unroll
          for (int i = 0; i < C::kCols / 4; ++i) {
            uint4 o;
            unpack2(acc[2 * i], o.x, o.y);
            unpack2(acc[2 * i + 1], o.z, o.w);
            st_cluster_u4(dst + i * 512, o);
          }
        }
        cluster_sync();
        if (owner != krank) break;
        if (rows > 0) {
          for (int r = 0; r + 1 < p.split; ++r) {
            const uint32_t src = slot(r);
#pragma unroll
            for (int i = 0; i < C::kCols / 4; ++i) {
              uint32_t v[4];
              lds_u4(src + i * 512, v);
              fma2(acc[2 * i], pack2(v[0], v[1]), dup2(1.f));
              fma2(acc[2 * i + 1], pack2(v[2], v[3]), dup2(1.f));
            }
          }
        }
      }
      if (!ok) break;
      if (rows <= 0) continue;
      // Through this warp's staging buffers (128-byte swizzle) to global memory: by TMA, or row
      // by row where the group ends inside the 32 rows.
      const int row = x.row0 + first;
#pragma unroll
      for (int ps = 0; ps < C::kCols / C::kPassCols; ++ps) {
        const int col = col0 + ps * C::kPassCols;
        if (col >= p.n_cols) break;
        const uint32_t stg = stg0 + (npass++ % C::kStgBufs) * 4096u;
        if (lane == 0) bulk_wait_group_read<C::kStgBufs - 1>();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 o;
          if constexpr (C::DW) {
            unpack2(acc[ps * 16 + 2 * c], o.x, o.y);
            unpack2(acc[ps * 16 + 2 * c + 1], o.z, o.w);
          } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack2(acc[ps * 32 + 4 * c + i], w[2 * i], w[2 * i + 1]);
            o.x = pack_bf16x2(__uint_as_float(w[0]), __uint_as_float(w[1]));
            o.y = pack_bf16x2(__uint_as_float(w[2]), __uint_as_float(w[3]));
            o.z = pack_bf16x2(__uint_as_float(w[4]), __uint_as_float(w[5]));
            o.w = pack_bf16x2(__uint_as_float(w[6]), __uint_as_float(w[7]));
          }
          sts_u4(stg + lane * 128u + ((uint32_t(c) ^ (lane & 7u)) << 4), o);
        }
        if (C::DW || rows == 32) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if constexpr (C::DW) tma_store_3d(&tmD, stg, col, row, x.e);
            else tma_store_2d(&tmD, stg, col, row);
          }
        } else {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + int(lane >> 3), c = int(lane & 7u);
            uint32_t v[4];
            lds_u4(stg + r * 128u + ((uint32_t(c) ^ (r & 7u)) << 4), v);
            if (r < rows && col + c * 8 < p.n_cols)
              *reinterpret_cast<uint4*>(p.d + int64_t(row + r) * p.ld_d + col + c * 8) =
                  make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        // (a group for every buffer, empty after plain stores, so that the wait above counts)
        if (lane == 0) bulk_commit_group();
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    if constexpr (C::SPLIT) {
      if (unit >= num_tiles) {      // no tile: the barriers that the others pass
        cluster_sync();
        cluster_sync();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (C::PAIR) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (C::PAIR) tmem_dealloc_pair(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

// --------------------------------------------------------------- host side

constexpr int kMaxDevices = 64;

// CTAs (single) or pairs that run at once on the current device; sets the kernel's
// shared-memory limit on the device's first use. 0 on failure.
template <class C>
int resident_units() {
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = cache[dev].load(std::memory_order_acquire);
  if (n > 0) return n;
  if (cudaFuncSetAttribute(expert_gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return 0;
  if (C::WIDE) {
    // The warpgroups' shares after the split have to fit in what the block is launched with:
    // one that asks for more would wait for good.
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, expert_gemm_kernel<C>) != cudaSuccess ||
        fa.numRegs * C::kThreads < C::kRoleRegs * 128 + C::kEpiRegs * 256)
      return 0;
  }
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 0;
  n = sms;
  if (C::PAIR) {
    cudaLaunchConfig_t qc = {};
    cudaLaunchAttribute qa[1];
    qa[0].id = cudaLaunchAttributeClusterDimension;
    qa[0].val.clusterDim.x = 2;
    qa[0].val.clusterDim.y = 1;
    qa[0].val.clusterDim.z = 1;
    qc.gridDim = dim3(sms / 2 * 2, 1, 1);
    qc.blockDim = dim3(C::kThreads, 1, 1);
    qc.dynamicSmemBytes = C::kSmem;
    qc.attrs = qa;
    qc.numAttrs = 1;
    n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, expert_gemm_kernel<C>, &qc) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = sms / 2;
    }
  }
  cache[dev].store(n, std::memory_order_release);
  return n;
}

// K steps of each CTA of a cluster that splits nk of them, in whole groups of four (e4m3's scales come
// four steps at a time): shares are rounded up, so the last CTAs may have fewer steps or none (33 steps
// over 4: 12, 12, 9, 0), and those without send zeros.
int split_part(int nk, int split) { return ((nk + split - 1) / split + 3) / 4 * 4; }

// Row tiles at most: every group may end inside a tile.
int64_t most_row_tiles(const ExpertArgs& a, int bm) {
  return std::min<int64_t>(a.M, (a.M + bm - 1) / bm + (a.offsets ? a.E - 1 : 0));
}

template <class C>
qlora_status launch_cfg(const ExpertArgs& a, cudaStream_t s, int split = 1) {
  const int max_units = resident_units<C>();
  if (max_units <= 0) return QLORA_ERR_CUDA;
  const TmapType ty = C::F8 ? TmapType::U8 : TmapType::BF16;
  const bool dw = C::DW, fwd = a.mode == ExpertMode::Fwd;
  const int64_t K = fwd ? a.in : a.out;         // Fwd, Dx: reduction length
  const int64_t N = fwd ? a.out : a.in;         // columns of D
  ExpertParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = int(a.M);
  p.E = int(a.E);
  p.n_cols = int(N);
  p.tiles_n = int((N + C::BN - 1) / C::BN);
  p.tiles_r = int((a.out + C::BM - 1) / C::BM);
  p.nk = int((K + C::BK - 1) / C::BK);
  p.split = split;
  p.k_part = split_part(p.nk, split);
  p.d_rows = int(a.out);
  // Groups of a few rows: boxes of 32 rows, so that a tile's unused rows are not fetched.
  p.a_box = (!C::PAIR && a.M < 64 * a.E) ? 32 : 128;
  p.offsets = a.offsets;
  p.sa = a.sa;
  p.sb = a.sb;
  p.nb_a = int((K + 127) / 128);
  p.sa_vec = p.nb_a % 4 == 0 && (reinterpret_cast<uintptr_t>(a.sa) & 15u) == 0;
  p.nb_n = int((N + 127) / 128);
  const int64_t nbo = (a.out + 127) / 128, nbi = (a.in + 127) / 128;
  p.sb_e = nbo * nbi;
  p.sb_n = fwd ? nbi : 1;
  p.sb_k = fwd ? 1 : nbi;
  p.d = static_cast<uint16_t*>(a.d);
  p.ld_d = N;
  p.status = a.status;

  CUtensorMap A, B, D;
  bool good;
  if (dw) {
    good = make_tmap_2d(&A, a.a, ty, a.out, a.M, a.out * C::kElem, 64, 64, true) &&
           make_tmap_2d(&B, a.b, ty, a.in, a.M, a.in * C::kElem, 64, 64, true) &&
           make_tmap_3d(&D, a.d, TmapType::F32, a.in, a.out, a.E, 32, 32);
  } else {
    good = make_tmap_2d(&A, a.a, ty, K, a.M, K * C::kElem, C::BK, p.a_box, true) &&
           make_tmap_3d(&B, a.b, ty, a.in, a.out, a.E, 128 / C::kElem, C::B_MN ? C::BK : 128) &&
           make_tmap_2d(&D, a.d, TmapType::BF16, N, a.M, N * 2, 64, 32, true);
  }
  if (!good) return QLORA_ERR_CUDA;

  const int64_t num_tiles = dw ? a.E * p.tiles_r * p.tiles_n : most_row_tiles(a, C::BM) * p.tiles_n;
  if (num_tiles > (int64_t(1) << 30)) return QLORA_ERR_SHAPE;
  // (SPLIT: one tile a cluster, however many run at once.)
  const int units = int(C::SPLIT ? num_tiles : std::min<int64_t>(num_tiles, max_units));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::PAIR ? 2 : unsigned(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(units * (C::PAIR ? 2 : split)), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  const int skip = pdl_enabled() ? 0 : 1;
  cfg.attrs = attr + skip;
  cfg.numAttrs = (C::PAIR || C::SPLIT ? 2 : 1) - skip;
  if (cudaLaunchKernelEx(&cfg, expert_gemm_kernel<C>, A, B, D, p) != cudaSuccess) {
    cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return QLORA_OK;
}

// The tile: by the time that the waves of tiles take, a wave's steps at the rates measured
// with full waves (us per step of 128 bytes of K; bf16 128 x 256 a tenth above its rate with
// operands in L2, for the weights of groups come from HBM):
//                  e4m3    bf16
//   128 x 128      0.33    0.27     148 at once; the most units and the fewest wasted rows
//   128 x 256      0.64    0.52     148 at once
//   256 x 256 pair 0.61    0.386    74 at once; half the L2 bytes of 128 x 128 per product
// (e4m3 4096 x 4096 at 512 rows: 12.6, 20.4 and 21.5 us; at 2048: 40.5, 39.5 and 40; at 8192:
// 148, 140 and 136. bf16 at 8192: 251, 207 and 173.) Groups' sizes are on the device: their row
// tiles are taken as half a tile more than full for each group, and the waves, where they
// are not safely one, as half a wave more (16 experts of 1408 x 2048 in bf16, 128 rows each
// on average: 25, 36 and 29 us; 64 of 1024 x 2048, 256 rows each: 99, 97 and 82).
// Dw, which writes fp32 and has few steps a tile, by the waves, a pair's a tenth shorter (16
// experts of 1408 x 2048, 512 rows each: 79, 76 and 71 us, waves of 20, 10 and 11; 64 of 1024 x
// 2048, 64 rows each: 116, 112 and 97 us, 28 waves of either).
// QLORA_B200_EXPERT_TILE=128|256|pair overrides the choice, for measurement and tests.
enum class ExpertTileKind { T128, T256, Pair };
template <bool F8>
ExpertTileKind tile_kind(const ExpertArgs& a) {
  const char* f = std::getenv("QLORA_B200_EXPERT_TILE");
  if (f) {
    if (std::strcmp(f, "128") == 0) return ExpertTileKind::T128;
    if (std::strcmp(f, "256") == 0) return ExpertTileKind::T256;
    if (std::strcmp(f, "pair") == 0) return ExpertTileKind::Pair;
  }
  if (a.mode == ExpertMode::Dw) {
    if (a.in <= 128) return ExpertTileKind::T128;
    auto waves = [&](int bm, int at_once) {
      return (a.E * ((a.out + bm - 1) / bm) * ((a.in + 255) / 256) + at_once - 1) / at_once;
    };
    return 9 * waves(256, 74) <= 10 * waves(128, 148) ? ExpertTileKind::Pair : ExpertTileKind::T256;
  }
  const int64_t N = a.mode == ExpertMode::Fwd ? a.out : a.in;
  auto cost = [&](int bm, int bn, int at_once, double step) {
    const int64_t cols = (N + bn - 1) / bn;
    if (!a.offsets) return double(((a.M + bm - 1) / bm * cols + at_once - 1) / at_once) * step;
    const double rows = std::max(double(std::min(a.E, a.M)), std::ceil(double(a.M) / bm) + 0.5 * double(a.E - 1));
    const double waves = rows * double(cols) / at_once;
    return (a.E == 1 ? std::ceil(waves) : waves <= 0.9 ? 1.0 : waves + 0.5) * step;
  };
  const double c128 = cost(128, 128, 148, F8 ? 0.33 : 0.27), c256 = cost(128, 256, 148, F8 ? 0.64 : 0.52),
               cpair = cost(256, 256, 74, F8 ? 0.61 : 0.386);
  if (cpair <= c256 && cpair <= c128) return ExpertTileKind::Pair;
  return c256 <= c128 ? ExpertTileKind::T256 : ExpertTileKind::T128;
}

// CTAs that share a 128 x 128 tile's K: where even the most tiles that there can be leave SMs
// idle, a share is eight steps or more, and all clusters run at once (16 of 8 CTAs do not: 22.9 us
// where 16 of 4 took 16.9, e4m3 at 256 rows, 1024 x 11008). e4m3 at 64 rows, 4096 x 4096: 9.7 us by four CTAs,
// 14.7 by one; 4096 x 11008: 17.1 and 35; at 256 rows by two: 13.4 and 15.9. bf16 at 17 rows,
// 4096 x 4096: 10.1 by four.
template <bool F8>
int split_of(const ExpertArgs& a) {
  const bool fwd = a.mode == ExpertMode::Fwd;
  const int64_t N = fwd ? a.out : a.in, K = fwd ? a.in : a.out;
  const int64_t tiles = most_row_tiles(a, 128) * ((N + 127) / 128);
  const int64_t nk = (K * (F8 ? 1 : 2) + 127) / 128;
  if (tiles <= 8 && nk >= 64) return 8;
  if (tiles <= 32 && nk >= 32) return 4;
  return tiles <= 74 && nk >= 16 ? 2 : 1;
}

template <bool F8, ExpertMode MODE>
qlora_status launch_mode(const ExpertArgs& a, cudaStream_t s) {
  switch (tile_kind<F8>(a)) {
    case ExpertTileKind::Pair: return launch_cfg<ExpertCfg<true, 256, F8, MODE>>(a, s);
    case ExpertTileKind::T256: return launch_cfg<ExpertCfg<false, 256, F8, MODE>>(a, s);
    default: break;
  }
  if constexpr (MODE != ExpertMode::Dw) {
    const int split = split_of<F8>(a);
    if (split > 1) return launch_cfg<ExpertCfg<false, 128, F8, MODE, true>>(a, s, split);
  }
  return launch_cfg<ExpertCfg<false, 128, F8, MODE>>(a, s);
}

}  // namespace

qlora_status launch_expert_gemm(const ExpertArgs& a, cudaStream_t s) {
  if (few_rows_wanted(a)) return launch_few_rows(a, false, s);
  switch (a.mode) {
    case ExpertMode::Fwd:
      return a.f8 ? launch_mode<true, ExpertMode::Fwd>(a, s) : launch_mode<false, ExpertMode::Fwd>(a, s);
    case ExpertMode::Dx:
      return a.f8 ? launch_mode<true, ExpertMode::Dx>(a, s) : launch_mode<false, ExpertMode::Dx>(a, s);
    case ExpertMode::Dw:
      return a.f8 ? QLORA_ERR_UNSUPPORTED : launch_mode<false, ExpertMode::Dw>(a, s);
  }
  return QLORA_ERR_UNSUPPORTED;
}

}  // namespace qlb
