// Quantizers to e4m3 with a scale for each 1 x 128 block of a row or each 128 x 128
// block of a weight. Bound by memory: 2 B read and 1 B written per value.
#include <algorithm>

#include "internal.cuh"
#include "block8.cuh"
#include "ptx.cuh"

namespace qlb {

namespace {

// 16 lanes per block of 128, 8 values a lane; a thread takes kRowIlp blocks, all loaded
// before the first is reduced.
constexpr int kRowThreads = 256, kRowIlp = 4;

// WHOLE: in % 128 == 0, so that block b starts at value 128 b (else a 64-bit division a block,
// which cost a third of the time: 30 us for 8192 x 4096 against 22).
template <bool WHOLE>
__global__ void __launch_bounds__(kRowThreads) quantize_rows8_kernel(const uint16_t* X, int64_t blocks,
                                                                     int64_t in, int64_t nb, uint8_t* codes,
                                                                     float* scale) {
  pdl_wait();
  pdl_launch();
  const int sub = threadIdx.x & 15;
  const int64_t b0 = int64_t(blockIdx.x) * (kRowThreads / 16 * kRowIlp) + (threadIdx.x >> 4);
  uint4 v[kRowIlp];
  int64_t at[kRowIlp];
#pragma unroll
  for (int j = 0; j < kRowIlp; ++j) {
    const int64_t b = b0 + j * (kRowThreads / 16);
    at[j] = -1;
    v[j] = make_uint4(0, 0, 0, 0);
    if (b < blocks) {
      if constexpr (WHOLE) {
        at[j] = b * 128 + sub * 8;
      } else {
        const int64_t row = b / nb;
        const int64_t col = (b - row * nb) * 128 + sub * 8;
        if (col < in) at[j] = row * in + col;
      }
      if (at[j] >= 0) v[j] = ld_global(reinterpret_cast<const uint4*>(X + at[j]));
    }
  }
#pragma unroll
  for (int j = 0; j < kRowIlp; ++j) {
    const int64_t b = b0 + j * (kRowThreads / 16);
    float f[8];
    bf16x8_to_f32(v[j], f);
    const Block8 q = block8_of(max16(max_abs8(v[j])));
    if (at[j] >= 0) *reinterpret_cast<uint2*>(codes + at[j]) = quantize8(f, q);
    if (b < blocks && sub == 0) scale[b] = q.scale;
  }
}

// One CTA per 128 x 128 block, held in registers between the maximum and the codes:
// thread t has the 8 columns 8 (t % 16).. of rows t / 16 + 16 j. 4096 x 4096: bf16 13.9 us, fp32 18.4 (the bytes
// take 7.7 and 12.8); two CTAs an SM and a barrier in each, so neither memory nor issue slots are full.
template <bool F32>
__global__ void __launch_bounds__(256) quantize_weight8_kernel(const void* W, int64_t out, int64_t in,
                                                               int64_t nb_in, int64_t nb_out, uint8_t* codes,
                                                               float* scale, int* status) {
  pdl_wait();
  pdl_launch();
  __shared__ uint32_t s_max[8];
  const int64_t blk = blockIdx.x;
  const int64_t bi = blk % nb_in, be = blk / nb_in;
  const int64_t bo = be % nb_out, e = be / nb_out;
  const int64_t col = bi * 128 + (threadIdx.x & 15) * 8;
  const int64_t row0 = bo * 128 + (threadIdx.x >> 4);
  const int64_t base = e * out * in;
  float f[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[j][i] = 0.f;
    const int64_t row = row0 + 16 * j;
    if (row < out && col < in) {
      if constexpr (F32) {
        const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(W) + base + row * in + col);
        const float4 a = ld_global(src), b = ld_global(src + 1);
        f[j][0] = a.x; f[j][1] = a.y; f[j][2] = a.z; f[j][3] = a.w;
        f[j][4] = b.x; f[j][5] = b.y; f[j][6] = b.z; f[j][7] = b.w;
      } else {
        bf16x8_to_f32(ld_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + base + row * in + col)),
                      f[j]);
      }
    }
    m = max(m, max_abs8(f[j]));
  }
  m = max16(m);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  const Block8 q = block8_of(m);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = row0 + 16 * j;
    if (row < out && col < in) *reinterpret_cast<uint2*>(codes + base + row * in + col) = quantize8<F32>(f[j], q);
  }
  if (threadIdx.x == 0) {
    scale[blk] = q.scale;
    if (m >= 0x7F800000u) set_status(status, QLORA_ERR_NONFINITE);
  }
}

}  // namespace

qlora_status launch_quantize_rows8(const uint16_t* X, int64_t M, int64_t in, uint8_t* codes, float* scale,
                                   cudaStream_t s) {
  const int64_t nb = (in + 127) / 128, blocks = M * nb;
  const int64_t per = kRowThreads / 16 * kRowIlp;
  const int64_t grid = (blocks + per - 1) / per;
  if (grid > 0x7FFFFFFF) return QLORA_ERR_SHAPE;
  const dim3 g = dim3(unsigned(grid)), t = dim3(kRowThreads);
  const cudaError_t r = in % 128 == 0
                            ? launch_pdl(quantize_rows8_kernel<true>, g, t, 0, s, X, blocks, in, nb, codes, scale)
                            : launch_pdl(quantize_rows8_kernel<false>, g, t, 0, s, X, blocks, in, nb, codes, scale);
  return r == cudaSuccess ? QLORA_OK : (cudaGetLastError(), QLORA_ERR_CUDA);
}

qlora_status launch_quantize_weight8(const void* W, bool f32, int64_t E, int64_t out, int64_t in, uint8_t* codes,
                                     float* scale, int* status, cudaStream_t s) {
  const int64_t nbi = (in + 127) / 128, nbo = (out + 127) / 128;
  const int64_t grid = E * nbi * nbo;
  if (grid > 0x7FFFFFFF) return QLORA_ERR_SHAPE;
  const cudaError_t r = f32 ? launch_pdl(quantize_weight8_kernel<true>, dim3(unsigned(grid)), dim3(256), 0, s, W, out,
                                         in, nbi, nbo, codes, scale, status)
                            : launch_pdl(quantize_weight8_kernel<false>, dim3(unsigned(grid)), dim3(256), 0, s, W, out,
                                         in, nbi, nbo, codes, scale, status);
  return r == cudaSuccess ? QLORA_OK : (cudaGetLastError(), QLORA_ERR_CUDA);
}

}  // namespace qlb
