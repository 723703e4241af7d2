// RMS norm of the residual stream, forward and backward.
//
//   h = bf16(x + r),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   g = dy w,  dx = dh + rstd (g - h rstd^2 mean(g h)),  dw = sum over rows of dy h rstd
//
// y leaves in bf16, in e4m3 with a scale for each 128 values (block8.cuh; quantized from
// the fp32 value, one rounding), or both. Sums, rstd and dw are fp32. Both directions
// are bound by memory: a row stays in registers between its sum and its output (in the backward up to
// H = 16384; above, 450 bytes a thread spill: with dw 1024 x 32768 takes 105 us, 2048 x 16384 64, 4096 x
// 8192 47). Each row is a CTA forward, of 32 threads at least: 131072 rows of 128 take 137 us, 4096 x 8192
// with twice the values 28.
#include <algorithm>

#include "internal.cuh"
#include "block8.cuh"
#include "nf4_device.cuh"
#include "ptx.cuh"

namespace qlb {

namespace {

// Sum over the CTA, the same bits in every thread (fixed order).
__device__ __forceinline__ float cta_sum(float v, float* s_part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = (threadIdx.x & 31) < warps ? s_part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
  return t;
}

template <bool F32>
__device__ __forceinline__ void load_w8(const void* w, int64_t col, float (&f)[8]) {
  if constexpr (F32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(w) + col);
    const float4 a = ld_global(src), b = ld_global(src + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    bf16x8_to_f32(ld_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + col)), f);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// One CTA per row; thread t holds the 8-value vectors t, t + T, ... (VPT of them), so 16
// neighbouring lanes hold one 128-value block.
template <int VPT, bool WF32>
__global__ void __launch_bounds__(512, VPT <= 2 ? 3 : 1) rms_norm_fwd_kernel(NormFwd a) {
  __shared__ float s_part[32];
  const int T = blockDim.x, nv = int(a.H >> 3);
  const int64_t row = blockIdx.x;
  pdl_wait();
  pdl_launch();
  uint4 v[VPT];
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + row * a.H);
  const uint4* rr = a.residual ? reinterpret_cast<const uint4*>(a.residual + row * a.H) : nullptr;
  uint4 r[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = int(threadIdx.x) + j * T;
    v[j] = i < nv ? ld_global(xr + i) : make_uint4(0, 0, 0, 0);
    r[j] = (rr && i < nv) ? ld_global(rr + i) : make_uint4(0, 0, 0, 0);
  }
  uint4 wv[VPT];
  if constexpr (!WF32) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = int(threadIdx.x) + j * T;
      wv[j] = i < nv ? ld_global(reinterpret_cast<const uint4*>(a.w) + i) : make_uint4(0, 0, 0, 0);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (rr) {
      float f[8], g[8];
      bf16x8_to_f32(v[j], f);
      bf16x8_to_f32(r[j], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] += g[k];
      v[j] = pack8(f);
    }
    float f[8];
    bf16x8_to_f32(v[j], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(f[k], f[k], ss);
    const int i = int(threadIdx.x) + j * T;
    if (a.h && i < nv) reinterpret_cast<uint4*>(a.h + row * a.H)[i] = v[j];
  }
  ss = cta_sum(ss, s_part);
  const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(ss, float(a.H)) + a.eps));
  if (threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int i = int(threadIdx.x) + j * T;
    float f[8], w[8];
    bf16x8_to_f32(v[j], f);
    if (i < nv) {
      if constexpr (WF32) load_w8<WF32>(a.w, int64_t(i) * 8, w);
      else bf16x8_to_f32(wv[j], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = f[k] * rstd * w[k];
      if (a.y) reinterpret_cast<uint4*>(a.y + row * a.H)[i] = pack8(f);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = 0.f;
    }
    if (a.y8 && j * T < nv) {       // whole warps: T and the bound are the same for all lanes
      const Block8 q = block8_of(max16(max_abs8(f)));
      if (i < nv) {
        reinterpret_cast<uint2*>(a.y8 + row * a.H)[i] = quantize8(f, q);
        if ((threadIdx.x & 15) == 0) a.y_scale[row * ((a.H + 127) >> 7) + (i >> 4)] = q.scale;
      }
    }
  }
}

// CTA c takes rows c, c + G, ...; its share of dw stays in registers and leaves as one
// row of partial sums, which rms_norm_dw_kernel adds in order.
template <int VPT, bool WF32>
__global__ void __launch_bounds__(512) rms_norm_bwd_kernel(NormBwd a) {
  __shared__ float s_part[2][32];
  const int T = blockDim.x, nv = int(a.H >> 3);
  pdl_wait();
  pdl_launch();
  float dw[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = 0.f;
  const float inv_h = __fdiv_rn(1.f, float(a.H));
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, flip ^= 1) {
    uint4 vy[VPT], vh[VPT], vd[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = int(threadIdx.x) + j * T;
      const uint4 z = make_uint4(0, 0, 0, 0);
      vy[j] = i < nv ? ld_global(reinterpret_cast<const uint4*>(a.dy + row * a.H) + i) : z;
      vh[j] = i < nv ? ld_global(reinterpret_cast<const uint4*>(a.h + row * a.H) + i) : z;
      vd[j] = (a.dh && i < nv) ? ld_global(reinterpret_cast<const uint4*>(a.dh + row * a.H) + i) : z;
    }
    const float rstd = ld_global(a.rstd + row);
    float c = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = int(threadIdx.x) + j * T;
      if (i < nv) {
        float y[8], h[8], w[8];
        bf16x8_to_f32(vy[j], y);
        bf16x8_to_f32(vh[j], h);
        load_w8<WF32>(a.w, int64_t(i) * 8, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float n = h[k] * rstd;
          dw[j][k] = fmaf(y[k], n, dw[j][k]);
          c = fmaf(y[k] * w[k], n, c);
        }
      }
    }
    c = cta_sum(c, s_part[flip]) * inv_h;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = int(threadIdx.x) + j * T;
      if (i < nv) {
        float y[8], h[8], w[8], d[8];
        bf16x8_to_f32(vy[j], y);
        bf16x8_to_f32(vh[j], h);
        bf16x8_to_f32(vd[j], d);
        load_w8<WF32>(a.w, int64_t(i) * 8, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = fmaf(rstd, fmaf(-h[k] * rstd, c, y[k] * w[k]), d[k]);
        reinterpret_cast<uint4*>(a.dx + row * a.H)[i] = pack8(d);
      }
    }
  }
  if (a.dw) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = int(threadIdx.x) + j * T;
      if (i < nv) {
        float4* dst = reinterpret_cast<float4*>(a.part + int64_t(blockIdx.x) * a.H) + 2 * i;
        dst[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        dst[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
      }
    }
  }
}

// dw[c] = the partial rows' sum: 32 columns x 32 row groups per CTA, groups added in order.
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float* part, int rows, int H,
                                                           float* dw) {
  __shared__ float s[32][33];
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int r = g; r < rows; r += 32) v += part[int64_t(r) * H + c];
  }
  s[g][lane] = v;
  __syncthreads();
  // warp g adds column g's groups: a fixed tree
  v = s[lane][g];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int col = blockIdx.x * 32 + g;
  if (lane == 0 && col < H) dw[col] = v;
}

struct NormShape {
  int threads, vpt;
};
// Two vectors a thread up to 512 threads (H = 8192), then more.
NormShape norm_shape(int64_t H) {
  const int nv = int(H / 8);
  NormShape n;
  n.threads = std::min(512, std::max(32, (((nv + 1) / 2) + 31) / 32 * 32));
  n.vpt = (nv + n.threads - 1) / n.threads;
  n.vpt = n.vpt <= 1 ? 1 : n.vpt <= 2 ? 2 : n.vpt <= 4 ? 4 : 8;
  return n;
}

template <bool WF32>
cudaError_t fwd_of(const NormFwd& a, cudaStream_t s) {
  const NormShape n = norm_shape(a.H);
  const dim3 grid = dim3(unsigned(a.M)), block = dim3(unsigned(n.threads));
  switch (n.vpt) {
    case 1: return launch_pdl(rms_norm_fwd_kernel<1, WF32>, grid, block, 0, s, a);
    case 2: return launch_pdl(rms_norm_fwd_kernel<2, WF32>, grid, block, 0, s, a);
    case 4: return launch_pdl(rms_norm_fwd_kernel<4, WF32>, grid, block, 0, s, a);
    default: return launch_pdl(rms_norm_fwd_kernel<8, WF32>, grid, block, 0, s, a);
  }
}

template <bool WF32>
cudaError_t bwd_of(const NormBwd& a, cudaStream_t s) {
  const NormShape n = norm_shape(a.H);
  const dim3 grid = dim3(unsigned(norm_bwd_parts(a.M, a.H))), block = dim3(unsigned(n.threads));
  switch (n.vpt) {
    case 1: return launch_pdl(rms_norm_bwd_kernel<1, WF32>, grid, block, 0, s, a);
    case 2: return launch_pdl(rms_norm_bwd_kernel<2, WF32>, grid, block, 0, s, a);
    case 4: return launch_pdl(rms_norm_bwd_kernel<4, WF32>, grid, block, 0, s, a);
    default: return launch_pdl(rms_norm_bwd_kernel<8, WF32>, grid, block, 0, s, a);
  }
}

}  // namespace

// CTAs of the backward (fixed, so that dw does not depend on the device).
int norm_bwd_parts(int64_t M, int64_t H) {
  const int threads = norm_shape(H).threads;
  const int per_sm = std::max(1, std::min(16, 1024 / threads));
  return int(std::min<int64_t>(M, int64_t(148) * per_sm));
}

qlora_status launch_rms_norm_fwd(const NormFwd& a, cudaStream_t s) {
  return (a.w_f32 ? fwd_of<true>(a, s) : fwd_of<false>(a, s)) == cudaSuccess ? QLORA_OK
                                                                            : (cudaGetLastError(), QLORA_ERR_CUDA);
}

qlora_status launch_rms_norm_bwd(const NormBwd& a, cudaStream_t s) {
  cudaError_t r = a.w_f32 ? bwd_of<true>(a, s) : bwd_of<false>(a, s);
  if (r == cudaSuccess && a.dw)
    r = launch_pdl(rms_norm_dw_kernel, dim3(unsigned((a.H + 31) / 32)), dim3(1024), 0, s, (const float*)a.part,
                   norm_bwd_parts(a.M, a.H), int(a.H), a.dw);
  return r == cudaSuccess ? QLORA_OK : (cudaGetLastError(), QLORA_ERR_CUDA);
}

}  // namespace qlb
