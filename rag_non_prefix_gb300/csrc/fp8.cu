// 8-bit floating point (e4m3) operators: the quantiser of rows and of weight blocks, and the
// RMS norm whose residual addition and quantisation run in the same pass.
//
// A group of channels (128 of one row, or a 128 x 128 block of a weight matrix) with largest
// magnitude a (at least 448 * 2^-126, so that neither a / 448 nor 448 / a leaves the normal
// fp32 numbers) has scale a / 448 and codes e4m3(x * (448 / a)): both quotients are IEEE fp32,
// the product is rounded once to fp32 (a value next to a border between two codes may therefore
// take the other one) and once to the nearest e4m3 number, ties to even, clamped at 448 (the
// product can round above it).  An infinity or a NaN in the group makes its largest magnitude
// infinite or NaN and every value of the group decode to NaN.
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace cb {

namespace {

__device__ __forceinline__ float fp8_amax_floor(uint32_t abs_bits) {
  // magnitudes compare as integers; NaN bits rank above infinity's, so a NaN survives the maximum
  return __uint_as_float(max(abs_bits, __float_as_uint(FP8_AMAX_MIN)));
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
template <int N> __device__ __forceinline__ uint32_t amax_bits(const float* f) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) m = max(m, abs_bits(f[j]));
  return m;
}
// maximum over the 16 lanes that hold one group
__device__ __forceinline__ uint32_t half_warp_max(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
__device__ __forceinline__ uint2 fp8_codes8(const float* f, float inv) {
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    h[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * inv, f[2 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// ----------------------------------------------------------------------------- rows
// One warp takes 256 channels of a row (16 lanes per group, 8 channels per lane), UNROLL rows at
// once so that their loads are in flight together.  Bound by HBM: (2 or 4) + 1 bytes per value.
constexpr int QR_UNROLL = 4;
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T* __restrict__ x, long long ldx, int rows, int cols,
                                                            uint8_t* __restrict__ codes, long long ldc,
                                                            float* __restrict__ scales, long long lds) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = (blockIdx.y * 256) + lane * 8;
  const long long row0 = (static_cast<long long>(blockIdx.x) * 8 + warp) * QR_UNROLL;
  const bool in = col < cols;
  float f[QR_UNROLL][8];
#pragma unroll
  for (int u = 0; u < QR_UNROLL; ++u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[u][j] = 0.f;
    if (in && row0 + u < rows) load8(x + (row0 + u) * ldx + col, f[u]);
  }
#pragma unroll
  for (int u = 0; u < QR_UNROLL; ++u) {
    const float a = fp8_amax_floor(half_warp_max(amax_bits<8>(f[u])));
    if (in && row0 + u < rows) {
      *reinterpret_cast<uint2*>(codes + (row0 + u) * ldc + col) = fp8_codes8(f[u], FP8_MAX / a);
      if ((lane & 15) == 0) scales[static_cast<long long>(col >> 7) * lds + row0 + u] = a / FP8_MAX;
    }
  }
}

// ----------------------------------------------------------------------------- weight blocks
// One CTA per 128 x 128 block, held in registers between the maximum and the codes (one read):
// a half warp per row segment of 128 channels, 8 rows per thread.
template <typename T>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const T* __restrict__ x, long long ldx, int rows, int cols,
                                                              uint8_t* __restrict__ codes, long long ldc,
                                                              float* __restrict__ scales, long long lds) {
  pdl_trigger();
  pdl_wait();
  __shared__ uint32_t red[8];
  const int t = threadIdx.x;
  const int col = blockIdx.x * 128 + (t & 15) * 8;
  const long long row = static_cast<long long>(blockIdx.y) * 128 + (t >> 4);
  const bool in = col < cols;
  float f[8][8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[u][j] = 0.f;
    if (in && row + u * 16 < rows) load8(x + (row + u * 16) * ldx + col, f[u]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) m = max(m, amax_bits<8>(f[u]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((t & 31) == 0) red[t >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, red[w]);
  const float a = fp8_amax_floor(m), inv = FP8_MAX / a;
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (in && row + u * 16 < rows)
      *reinterpret_cast<uint2*>(codes + (row + u * 16) * ldc + col) = fp8_codes8(f[u], inv);
  if (t == 0) scales[static_cast<long long>(blockIdx.y) * lds + blockIdx.x] = a / FP8_MAX;
}

// ----------------------------------------------------------------------------- norm
// One CTA per row, the row held in registers from its single read to its codes: thread t owns
// the 8-channel pieces t, t + blockDim, ... (CH of them), so 16 consecutive lanes hold one group.
// h = residual + x in fp32; the norm and the codes come from the unrounded h, residual_out gets h
// rounded to its type.
template <typename TX, typename TR, int CH>
__global__ void __launch_bounds__(1024) add_rmsnorm_fp8_kernel(const TX* __restrict__ x, long long ldx,
                                                               const TR* res, TR* res_out, long long ldr,
                                                               const TX* __restrict__ weight, int d, float eps,
                                                               uint8_t* __restrict__ codes, long long ldc,
                                                               float* __restrict__ scales, long long lds) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[32];
  const long long row = blockIdx.x;
  const int t = threadIdx.x, T = blockDim.x;
  float f[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (t + k * T) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[k][j] = 0.f;
    if (c < d) load8(x + row * ldx + c, f[k]);
  }
  if (res) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = (t + k * T) * 8;
      if (c < d) {
        float r[8];
        load8(res + row * ldr + c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[k][j] = r[j] + f[k][j];
        if (res_out) store8(res_out + row * ldr + c, f[k]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += f[k][j] * f[k][j];
  ss = warp_sum(ss);
  if ((t & 31) == 0) red[t >> 5] = ss;
  __syncthreads();
  const int nw = T >> 5;
  ss = warp_sum((t & 31) < nw ? red[t & 31] : 0.f);
  const float inv_rms = 1.0f / sqrtf(ss / static_cast<float>(d) + eps);
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (t + k * T) * 8;
    if (weight && c < d) {
      float w[8];
      load8(weight + c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[k][j] *= w[j];
    }
    // y = u * inv_rms with u = h * w, so y * (448 / max|y|) = u * (448 / max|u|): the codes do not
    // see the norm's rounding (two roundings instead of four), only the scale does.  Where 448 /
    // max|u| could overflow, or the scale's floor applies, the codes come from y itself.
    const float au = __uint_as_float(half_warp_max(amax_bits<8>(f[k])));
    const float a = fp8_amax_floor(abs_bits(au * inv_rms));
    float inv = FP8_MAX / au;
    if (!(au > 0x1p-100f && a > FP8_AMAX_MIN)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[k][j] *= inv_rms;
      inv = FP8_MAX / a;
    }
    if (c < d) {
      *reinterpret_cast<uint2*>(codes + row * ldc + c) = fp8_codes8(f[k], inv);
      if ((t & 15) == 0) scales[static_cast<long long>(c >> 7) * lds + row] = a / FP8_MAX;
    }
  }
}

template <typename TX, typename TR>
cudaError_t launch_norm(const void* x, long long ldx, const void* res, void* res_out, long long ldr, const void* weight,
                        int rows, int d, float eps, void* codes, long long ldc, float* scales, long long lds,
                        cudaStream_t s) {
  // threads of a row in whole warps, one piece of 8 channels each
  const int pieces = (d + 7) / 8;
  auto go = [&](auto kernel, int ch) {
    const int threads = ((pieces + ch - 1) / ch + 31) / 32 * 32;
    return launch_chain(kernel, dim3(rows), dim3(threads), 0, s, static_cast<const TX*>(x), ldx,
                        static_cast<const TR*>(res), static_cast<TR*>(res_out), ldr, static_cast<const TX*>(weight), d,
                        eps, static_cast<uint8_t*>(codes), ldc, scales, lds);
  };
  return go(add_rmsnorm_fp8_kernel<TX, TR, 4>, 4);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* x, long long ldx, int rows, int cols, cb_dtype dt, int block_rows,
                                void* codes, long long ldc, float* scales, long long lds, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  uint8_t* c = static_cast<uint8_t*>(codes);
  if (block_rows == 1) {
    const dim3 grid((rows + 8 * QR_UNROLL - 1) / (8 * QR_UNROLL), (cols + 255) / 256);
    if (dt == CB_BF16)
      return launch_chain(quantize_rows_kernel<bf16>, grid, dim3(256), 0, s, static_cast<const bf16*>(x), ldx, rows, cols,
                          c, ldc, scales, lds);
    return launch_chain(quantize_rows_kernel<float>, grid, dim3(256), 0, s, static_cast<const float*>(x), ldx, rows, cols,
                        c, ldc, scales, lds);
  }
  const dim3 grid((cols + 127) / 128, (rows + 127) / 128);
  if (dt == CB_BF16)
    return launch_chain(quantize_blocks_kernel<bf16>, grid, dim3(256), 0, s, static_cast<const bf16*>(x), ldx, rows, cols,
                        c, ldc, scales, lds);
  return launch_chain(quantize_blocks_kernel<float>, grid, dim3(256), 0, s, static_cast<const float*>(x), ldx, rows, cols,
                      c, ldc, scales, lds);
}

cudaError_t launch_add_rmsnorm_fp8(const void* x, long long ldx, cb_dtype xdt, const void* res, void* res_out,
                                   long long ldr, cb_dtype rdt, const void* weight, int rows, int d, float eps,
                                   void* codes, long long ldc, float* scales, long long lds, cudaStream_t s) {
  if (rows <= 0) return cudaSuccess;
  if (xdt == CB_BF16)
    return rdt == CB_BF16
               ? launch_norm<bf16, bf16>(x, ldx, res, res_out, ldr, weight, rows, d, eps, codes, ldc, scales, lds, s)
               : launch_norm<bf16, float>(x, ldx, res, res_out, ldr, weight, rows, d, eps, codes, ldc, scales, lds, s);
  return rdt == CB_BF16
             ? launch_norm<float, bf16>(x, ldx, res, res_out, ldr, weight, rows, d, eps, codes, ldc, scales, lds, s)
             : launch_norm<float, float>(x, ldx, res, res_out, ldr, weight, rows, d, eps, codes, ldc, scales, lds, s);
}

}  // namespace cb
