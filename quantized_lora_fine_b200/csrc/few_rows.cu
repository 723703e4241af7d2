// Y_e = X_e W_e^T for few rows a group (decoding): bound by reading the weights once.
//
// A CTA takes 16 rows of one expert's weight over all of K, its 4, 8 or 16 warps every fourth,
// eighth or sixteenth 128-byte block of K. The rows stream from global memory into the registers of
// mma.sync fragments: lane (g, t) loads bytes 16 t .. and 64 + 16 t .. of weight rows g and
// g + 8 and of token g, and gives their words to four products in the same order on both
// sides (a sum over k may run over k in any order), so every load is 16 bytes wide, a warp's
// cover whole sectors and nothing passes through shared memory. Weight rows are the
// product's 16 rows, tokens its 8 columns. In e4m3 a block's product is scaled by sa sb and
// added in fp32; the warps' sums are added in order at the end. 32 experts of 2048 x 4096, 4 rows
// on average: bf16 81 us, e4m3 45 (its products go through 16-bit ones).
// (e4m3 weights by cp.async into shared memory, 4 blocks ahead: 64 us for 51 then.)
//
// A CTA makes one pass of 8 rows over its own expert's weight rows. Groups with more rows have later
// passes; they are one list, dealt out to the first CTAs, one each, so that no CTA makes more than two
// passes however the rows are routed. (An expert's own CTAs for all of its passes: with all rows in
// one of 32 experts of 2048 x 4096, 128 rows took 115 us in bf16 and 79 in e4m3 for 35 and 22; in one of 1024 of
// 256 x 256, 4096 rows took 438 and 362 for 75 and 50. Evenly routed: 84 and 48 us for 84 and 47, and 61
// and 34 for 66 and 35.)
//
// With bf16 rows and an e4m3 weight (QUANT, up to 2 rows in all) each warp quantizes the
// blocks that it multiplies, as quantize_rows8_kernel does, which saves that launch (every
// CTA quantizes every row: at 8 rows that took longer than the launch).
//
// tcgen05 tiles of 128 rows would leave most SMs without a tile here: 4096 x 4096 has 32.
#include <algorithm>
#include <cstdlib>

#include "block8.cuh"
#include "expert_gemm.cuh"
#include "internal.cuh"
#include "nf4_device.cuh"
#include "ptx.cuh"

namespace qlb {

namespace {

struct FewParams {
  const uint8_t* w;      // [E][out][wbytes]
  const uint8_t* x;      // [M][wbytes], or bf16 [M][in] with QUANT
  const float* sa;
  const float* sb;
  const int32_t* offsets;
  uint16_t* y;
  int* status;
  int M, E, out, in;
  int wbytes;            // bytes of a weight row
  int nk;                // 128-byte blocks of K
  int nb_n;              // scale rows per expert
};

template <bool F8>
__device__ __forceinline__ void mma16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  if constexpr (F8) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// 16 bytes at p and 16 at p + 64; zero where the row ends (at a multiple of 16; `left` from p).
__device__ __forceinline__ void load32(uint32_t (&v)[8], const uint8_t* p, int left) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  const uint4 a = left >= 16 ? ld_global(reinterpret_cast<const uint4*>(p)) : z;
  const uint4 b = left >= 80 ? ld_global(reinterpret_cast<const uint4*>(p) + 4) : z;
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// Weights are read once: not kept in L1.
__device__ __forceinline__ void stream32(uint32_t (&v)[8], const uint8_t* p, int left) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  const uint4 a = left >= 16 ? ld_stream(reinterpret_cast<const uint4*>(p)) : z;
  const uint4 b = left >= 80 ? ld_stream(reinterpret_cast<const uint4*>(p) + 4) : z;
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Pass `y` of the list of all groups' passes but their first, ROWS rows each (a group's last has what is
// left), found by the whole warp, 128 groups at a time, four a lane: its expert, its first row and the end
// of its group. False past the list's end.
template <int ROWS>
__device__ __forceinline__ bool later_pass(const FewParams& p, int y, int lane, int& e, int& m0, int& last) {
  int run = 0, before = 0;                        // the running maximum, and the passes, of the groups so far
  for (int c = 0; c < p.E; c += 128) {
    const int b = c + lane * 4;
    int s[5];                                     // starts of the lane's groups and the last one's end
#pragma unroll
    for (int j = 0; j < 5; ++j) s[j] = min(max(ld_global(p.offsets + min(b + j, p.E)), 0), p.M);
    int top = max(max(s[0], s[1]), max(s[2], s[3]));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, top, d);
      if (lane >= d) top = max(top, u);
    }
    const int left = __shfl_up_sync(0xffffffffu, top, 1);
    s[0] = max(s[0], lane == 0 ? run : max(run, left));
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j + 1] = max(s[j], s[j + 1]);
      n += max(s[j + 1] - s[j] - 1, 0) / ROWS;
    }
    int upto = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += u;
    }
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    if (y < before + all) {
      int k = y - before - (upto - n);            // in 0 .. n - 1 for the lane that has it
      const uint32_t who = __ballot_sync(0xffffffffu, k >= 0 && k < n);
      bool found = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int of = max(s[j + 1] - s[j] - 1, 0) / ROWS;
        if (!found && k < of) {
          found = true;
          e = b + j;
          m0 = s[j] + (k + 1) * ROWS;
          last = s[j + 1];
        }
        k -= of;
      }
      const int src = __ffs(int(who)) - 1;
      e = __shfl_sync(0xffffffffu, e, src);
      m0 = __shfl_sync(0xffffffffu, m0, src);
      last = __shfl_sync(0xffffffffu, last, src);
      return true;
    }
    before += all;
    run = max(run, __shfl_sync(0xffffffffu, top, 31));
  }
  return false;
}

// NT: 8-token columns a pass; U: blocks of K in flight a warp; WARPS a CTA, CTAS an SM. GROUPS: rows by
// offsets; else all rows (one pass) go through one weight.
template <bool F8, int NT, int U, bool GROUPS, bool QUANT, int WARPS, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS) few_rows_kernel(const FewParams p) {
  static_assert(kFewQuantRows == 2, "tokens 0 and 1 are lane t = 0's");
  static_assert(!QUANT || (F8 && NT == 1 && U == 1 && !GROUPS), "rows quantized here: kFewQuantRows, in e4m3");
  __shared__ float red[WARPS][NT * 8][17];
  __shared__ int s_later[WARPS];
  __shared__ __align__(16) uint8_t xq[QUANT ? WARPS * kFewQuantRows * 128 : 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  constexpr int ROWS = NT * 8;
  const int n0 = blockIdx.x * 16;
  int e = blockIdx.y;
  pdl_wait();
  pdl_launch();
  // The group's rows: the running maximum of the offsets clamped to [0, M], as the tiled kernel.
  int m0 = 0, last = p.M;
  // Passes beyond their groups' first go to the first CTAs, one each: there are (M - 1) / ROWS at most.
  const bool helps = GROUPS && int(blockIdx.y) < (p.M - 1) / ROWS;
  if constexpr (GROUPS) {
    const int i0 = helps ? int(threadIdx.x) : p.E;
    const int o0 = i0 < p.E ? ld_global(p.offsets + i0) : 0, o1 = i0 < p.E ? ld_global(p.offsets + i0 + 1) : 0;
    int v = 0;
    for (int i = lane; i <= e; i += 32) v = max(v, ld_global(p.offsets + i));
    const int r0 = ld_global(p.offsets + e), r1 = ld_global(p.offsets + e + 1);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
    m0 = min(v, p.M);
    last = max(m0, min(max(r1, 0), p.M));
    if (blockIdx.x == 0 && threadIdx.x == 0 && (r0 < 0 || r1 > p.M || r1 < r0))
      set_status_site(p.status, QLORA_ERR_SHAPE, 70);
    if (helps) {                                   // how many (at least as many where the offsets descend)
      auto beyond = [&](int from, int to) {
        return max(min(max(to, 0), p.M) - min(max(from, 0), p.M) - 1, 0) / ROWS;
      };
      int n = beyond(o0, o1);
      for (int i = i0 + WARPS * 32; i < p.E; i += WARPS * 32)
        n += beyond(ld_global(p.offsets + i), ld_global(p.offsets + i + 1));
      n = int(__reduce_add_sync(0xffffffffu, unsigned(n)));
      if (lane == 0) s_later[warp] = n;
    }
  }
  // After a barrier: the next of the groups' later passes for this CTA, if there is one. (A group that has most of
  // the rows would keep its own CTAs for a pass after another.)
  int y = blockIdx.y;
  auto next = [&]() {
    int n = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) n += s_later[i];
    if (y >= n || !later_pass<ROWS>(p, y, lane, e, m0, last)) return false;
    y += gridDim.y;
    return true;
  };
  if (GROUPS && m0 >= last) {
    if (!helps) return;
    __syncthreads();
    if (!next()) return;
  }
  for (;;) {
    const uint8_t* w0 = p.w + (int64_t(e) * p.out + n0 + g) * p.wbytes + 16 * t;
    const uint8_t* w1 = w0 + int64_t(8) * p.wbytes;
    const float* sb = F8 ? p.sb + (int64_t(e) * p.nb_n + (n0 >> 7)) * p.nk : nullptr;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    uint2 xv[kFewQuantRows];                       // QUANT: the next block of every row, 4 values a lane
    auto fetch = [&](int k) {
      const int col = k * 128 + lane * 4;
#pragma unroll
      for (int m = 0; m < kFewQuantRows; ++m)
        xv[m] = (m0 + m < last && col < p.in)
                    ? ld_global(reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p.x) +
                                                           int64_t(m0 + m) * p.in + col))
                    : make_uint2(0, 0);
    };
    if constexpr (QUANT) fetch(warp);
    for (int k0 = warp; k0 < p.nk; k0 += WARPS * U) {
      uint32_t a[U][2][8], b[U][NT][8];
      float f[U][NT][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * WARPS;
        const int left = k < p.nk ? p.wbytes - k * 128 - 16 * t : 0;
        stream32(a[u][0], w0 + int64_t(k) * 128, left);
        stream32(a[u][1], w1 + int64_t(k) * 128, left);
      }
      float xs[2] = {0.f, 0.f};                    // QUANT: scales of tokens 2 t, 2 t + 1
      if constexpr (QUANT) {
        // this block of every row to codes in the warp's own shared memory
        uint8_t* xw = xq + warp * kFewQuantRows * 128;
        uint2 v[kFewQuantRows];
#pragma unroll
        for (int m = 0; m < kFewQuantRows; ++m) v[m] = xv[m];
        fetch(k0 + WARPS);
        __syncwarp();
#pragma unroll
        for (int m = 0; m < kFewQuantRows; ++m) {
          uint32_t mx = max(max(v[m].x & 0x7FFFu, (v[m].x >> 16) & 0x7FFFu),
                            max(v[m].y & 0x7FFFu, (v[m].y >> 16) & 0x7FFFu)) << 16;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          const Block8 q = block8_of(mx);
          reinterpret_cast<uint32_t*>(xw + m * 128)[lane] =
              e4m3x4(block8_quotient(__uint_as_float(v[m].x << 16), q),
                     block8_quotient(__uint_as_float(v[m].x & 0xFFFF0000u), q),
                     block8_quotient(__uint_as_float(v[m].y << 16), q),
                     block8_quotient(__uint_as_float(v[m].y & 0xFFFF0000u), q));
          if (t == 0) xs[m] = q.scale;
        }
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * WARPS;
        const int left = k < p.nk ? p.wbytes - k * 128 - 16 * t : 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int m = m0 + n * 8 + g;
          if constexpr (QUANT) {
            const uint8_t* src = xq + (warp * kFewQuantRows + (g & 1)) * 128 + 16 * t;
            const bool live = g < kFewQuantRows && m < last;
            const uint4 z = make_uint4(0, 0, 0, 0);
            const uint4 lo = live ? reinterpret_cast<const uint4*>(src)[0] : z;
            const uint4 hi = live ? reinterpret_cast<const uint4*>(src)[4] : z;
            b[u][n][0] = lo.x; b[u][n][1] = lo.y; b[u][n][2] = lo.z; b[u][n][3] = lo.w;
            b[u][n][4] = hi.x; b[u][n][5] = hi.y; b[u][n][6] = hi.z; b[u][n][7] = hi.w;
          } else {
            load32(b[u][n], p.x + int64_t(m) * p.wbytes + k * 128 + 16 * t, m < last ? left : 0);
          }
          if constexpr (F8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = m0 + n * 8 + 2 * t + h;
              f[u][n][h] = 0.f;
              if (c < last && k < p.nk) {
                if constexpr (QUANT) f[u][n][h] = xs[h] * ld_global(sb + k);
                else f[u][n][h] = ld_global(p.sa + int64_t(c) * p.nk + k) * ld_global(sb + k);
              }
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (F8) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma16x8<F8>(c, a[u][0][2 * j], a[u][1][2 * j], a[u][0][2 * j + 1], a[u][1][2 * j + 1], b[u][n][2 * j],
                          b[u][n][2 * j + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = fmaf(c[i], f[u][n][i & 1], acc[n][i]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma16x8<F8>(acc[n], a[u][0][2 * j], a[u][1][2 * j], a[u][0][2 * j + 1], a[u][1][2 * j + 1],
                          b[u][n][2 * j], b[u][n][2 * j + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][n * 8 + 2 * t + (i & 1)][g + (i >> 1) * 8] = acc[n][i];
    __syncthreads();
    const int r = threadIdx.x & 15;
    for (int m = threadIdx.x >> 4; m < ROWS && m0 + m < last; m += WARPS * 2) {
      float s = red[0][m][r];
#pragma unroll
      for (int k = 1; k < WARPS; ++k) s += red[k][m][r];
      p.y[int64_t(m0 + m) * p.out + n0 + r] = uint16_t(pack_bf16x2(s, s) & 0xFFFFu);
    }
    if (!helps || !next()) return;
    __syncthreads();
  }
}

}  // namespace

// Up to 16 rows of one group, or 4 a group on average, 5 in bf16 (more rows are right, but each pass of 8
// fetches the weights again). 4096 x 4096 in e4m3 at 16 rows: 7.4 us against 9.6 with tiles (4096 x 11008:
// 15.7 and 14.8). 64 experts of 1024 x 2048 at four, five and eight rows a group: bf16 43, 44 and 53 us, tiles
// 47, 47 and 48; e4m3 28, 29 and 35, tiles 29, 29 and 30; 16 of 5120 x 5120: bf16 122, 129 and 163, tiles
// 142, 144 and 145; e4m3 74, 76 and 99, tiles 77, 79 and 79. With every row in one group a call takes no longer
// than with even groups, but tiles take less: 128 rows in one of 32 experts of 2048 x 4096, 35 us in bf16 and
// 22 in e4m3, tiles 20 and 14; 1024 in one of 256 of 768 x 2048, 64 and 45, tiles 19 and 16. The host does not see
// the groups' sizes. QLORA_B200_EXPERT_TILE set: never.
bool few_rows_wanted(const ExpertArgs& a) {
  if (a.mode != ExpertMode::Fwd || std::getenv("QLORA_B200_EXPERT_TILE")) return false;
  return a.offsets ? a.M <= (a.f8 ? 4 : 5) * a.E : a.M <= 16;
}

// Warps a CTA: 4 where the CTAs are many, for the sums at the end and the first loads of small CTAs
// overlap others' (64 experts of 1024 x 2048 at one and four rows a group: bf16 26 and 43 us, 8 warps
// 32 and 48; e4m3 17 and 28, 8 warps 20 and 31). More where there is no other CTA to overlap with: 16 in e4m3
// (4096 x 4096 5.3 us, 8 warps 6.2; 4096 x 11008 10.5 and 13.3; 2048 x 16384 11.4 and 16.9; 11008 x 4096, 688
// CTAs, 11.2 and 11.4), 8 in bf16 (one group of 4096 x 4096: 6.0 us, 4 warps 7.1). Two passes in one
// (9 to 16 rows): 16 warps where each CTA has an SM (2048 x 16384: 14 us, 8 warps 18.6; 4096 x 4096, which has
// more CTAs: 9.4 and 7.7).
qlora_status launch_few_rows(const ExpertArgs& a, bool quantize, cudaStream_t s) {
  FewParams p = {};
  p.w = static_cast<const uint8_t*>(a.b);
  p.x = static_cast<const uint8_t*>(a.a);
  p.sa = a.sa;
  p.sb = a.sb;
  p.offsets = a.offsets;
  p.y = static_cast<uint16_t*>(a.d);
  p.status = a.status;
  p.M = int(a.M);
  p.E = int(a.E);
  p.out = int(a.out);
  p.in = int(a.in);
  p.wbytes = int(a.in) * (a.f8 ? 1 : 2);
  p.nk = (p.wbytes + 127) / 128;
  p.nb_n = int((a.out + 127) / 128);
  const dim3 grid(unsigned(a.out / 16), unsigned(a.E));
  const int64_t ctas = int64_t(grid.x) * grid.y;
  auto launch = [&](auto* kernel, int warps) { return launch_pdl(kernel, grid, dim3(unsigned(warps * 32)), 0, s, p); };
  cudaError_t r;
  if (quantize) {
    r = launch(few_rows_kernel<true, 1, 1, false, true, 16, 2>, 16);
  } else if (!a.f8) {   // (bf16 rows always come in groups, a few each)
    r = ctas <= 148 * 2 ? launch(few_rows_kernel<false, 1, 4, true, false, 8, 2>, 8)
                        : launch(few_rows_kernel<false, 1, 4, true, false, 4, 4>, 4);
  } else if (!a.offsets && a.M > 8) {
    r = ctas <= 148 ? launch(few_rows_kernel<true, 2, 1, false, false, 16, 1>, 16)
                    : launch(few_rows_kernel<true, 2, 2, false, false, 8, 2>, 8);
  } else if (!a.offsets) {
    r = launch(few_rows_kernel<true, 1, 1, false, false, 16, 2>, 16);
  } else if (ctas <= 148 * 2) {
    r = launch(few_rows_kernel<true, 1, 1, true, false, 16, 2>, 16);
  } else {
    r = launch(few_rows_kernel<true, 1, 1, true, false, 4, 8>, 4);
  }
  return r == cudaSuccess ? QLORA_OK : (cudaGetLastError(), QLORA_ERR_CUDA);
}

}  // namespace qlb
