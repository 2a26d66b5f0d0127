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
// largest magnitude of three values, NaN if one is (one instruction on sm_100 and later)
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}
// largest magnitude of eight values as bits (NaN bits rank above infinity's)
__device__ __forceinline__ uint32_t amax_bits8(const float* f) {
  return __float_as_uint(max3_abs(max3_abs(f[0], f[1], f[2]), max3_abs(f[3], f[4], f[5]), max3_abs(f[6], f[7], 0.f)));
}
// 8 values as they lie in memory: 4 registers (bf16) or 8 (fp32)
template <typename T> struct Piece;
template <> struct Piece<bf16> {
  uint4 v = make_uint4(0, 0, 0, 0);
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint4*>(p); }
  // magnitudes of bf16 compare as 16-bit integers, two at once
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m & 0xffff0000u, m << 16);
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <> struct Piece<float> {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ uint32_t amax() const {
    float f[8];
    get(f);
    return amax_bits8(f);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
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
  Piece<T> v[QR_UNROLL];
#pragma unroll
  for (int u = 0; u < QR_UNROLL; ++u)
    if (in && row0 + u < rows) v[u].load(x + (row0 + u) * ldx + col);
#pragma unroll
  for (int u = 0; u < QR_UNROLL; ++u) {
    const float a = fp8_amax_floor(half_warp_max(v[u].amax()));
    if (in && row0 + u < rows) {
      float f[8];
      v[u].get(f);
      *reinterpret_cast<uint2*>(codes + (row0 + u) * ldc + col) = fp8_codes8(f, FP8_MAX / a);
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
  const unsigned groups = (cols + 127) / 128;
  const unsigned block = blockIdx.x / groups, group = blockIdx.x - block * groups;
  const int col = group * 128 + (t & 15) * 8;
  const long long row = static_cast<long long>(block) * 128 + (t >> 4);
  const bool in = col < cols;
  Piece<T> v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (in && row + u * 16 < rows) v[u].load(x + (row + u * 16) * ldx + col);
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) m = max(m, v[u].amax());
  m = __reduce_max_sync(0xffffffffu, m);
  if ((t & 31) == 0) red[t >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, red[w]);
  const float a = fp8_amax_floor(m), inv = FP8_MAX / a;
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (in && row + u * 16 < rows) {
      float f[8];
      v[u].get(f);
      *reinterpret_cast<uint2*>(codes + (row + u * 16) * ldc + col) = fp8_codes8(f, inv);
    }
  if (t == 0) scales[static_cast<long long>(block) * lds + group] = a / FP8_MAX;
}

// ----------------------------------------------------------------------------- norm
// A row is held in registers from its single read to its codes: thread t owns the 8-channel pieces
// t, t + blockDim, ... (CH of them), so 16 consecutive lanes hold one group.  h = residual + x in
// fp32; the norm and the codes come from the unrounded h, residual_out gets h rounded to its type.

// Sum over the block.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int n = blockDim.x >> 5;
  float sum = 0.f;
  for (int i = 0; i < n; ++i) sum += red[i];
  return sum;
}

// Codes and scales of the row h (in f), given 1 / rms.
template <typename TX, int CH>
__device__ __forceinline__ void norm_codes(float (&f)[CH][8], float inv_rms, const TX* __restrict__ weight, int d,
                                           long long row, uint8_t* __restrict__ codes, long long ldc,
                                           float* __restrict__ scales, long long lds) {
  const int t = threadIdx.x, T = blockDim.x;
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
    const float au = __uint_as_float(half_warp_max(amax_bits8(f[k])));
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

template <typename TX, typename TR, bool RES, int CH>
__global__ void __launch_bounds__(1024) add_rmsnorm_fp8_kernel(const TX* __restrict__ x, long long ldx,
                                                               const void* residual, void* residual_out, long long ldr,
                                                               const TX* __restrict__ weight, int d, float eps,
                                                               uint8_t* __restrict__ codes, long long ldc,
                                                               float* __restrict__ scales, long long lds) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[32];
  const TR* res = static_cast<const TR*>(residual);
  TR* res_out = static_cast<TR*>(residual_out);
  const long long row = blockIdx.x;
  const int t = threadIdx.x, T = blockDim.x;
  // every read is under way before the first value is needed (residual_out may be residual, so the
  // compiler may not move a read across its store)
  Piece<TX> px[CH];
  Piece<TR> pr[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (t + k * T) * 8;
    if (c < d) {
      px[k].load(x + row * ldx + c);
      if (RES) pr[k].load(res + row * ldr + c);
    }
  }
  float f[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (t + k * T) * 8;
    float r[8];
    px[k].get(f[k]);
    pr[k].get(r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (RES) f[k][j] = r[j] + f[k][j];
      ss += f[k][j] * f[k][j];
    }
    if (RES && res_out && c < d) store8(res_out + row * ldr + c, f[k]);
  }
  const float inv_rms = 1.0f / sqrtf(block_sum(ss, red) / static_cast<float>(d) + eps);
  norm_codes<TX, CH>(f, inv_rms, weight, d, row, codes, ldc, scales, lds);
}

template <typename TX, typename TR>
cudaError_t launch_norm(const void* x, long long ldx, const void* res, void* res_out, long long ldr, const void* weight,
                        int rows, int d, float eps, void* codes, long long ldc, float* scales, long long lds,
                        cudaStream_t s) {
  const int pieces = (d + 7) / 8;
  auto one = [&](auto kernel, int ch) {
    const int threads = ((pieces + ch - 1) / ch + 31) / 32 * 32;
    return launch_chain(kernel, dim3(rows), dim3(threads), 0, s, static_cast<const TX*>(x), ldx,
                        res, res_out, ldr, static_cast<const TX*>(weight), d, eps, static_cast<uint8_t*>(codes), ldc, scales, lds);
  };
  // Pieces per thread: one for short rows and for few rows (the shortest way through a row: 2.4 us for
  // one row of 4096 against 3.2 us with four; 2000 rows of 1024: 5.0 against 6.5 us), four for many
  // long ones, whose CTAs then keep more reads under way per barrier (8320 rows of 8192 in bf16: 78
  // against 97 us; 8320 rows of 7168 with an fp32 residual: 99 against 106 us).
  const bool one_piece = pieces <= 1024 && (pieces <= 512 || rows <= 608);
  if (res) return one_piece ? one(add_rmsnorm_fp8_kernel<TX, TR, true, 1>, 1) : one(add_rmsnorm_fp8_kernel<TX, TR, true, 4>, 4);
  return one_piece ? one(add_rmsnorm_fp8_kernel<TX, TX, false, 1>, 1) : one(add_rmsnorm_fp8_kernel<TX, TX, false, 4>, 4);
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
  const long long blocks = static_cast<long long>((cols + 127) / 128) * ((rows + 127) / 128);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks));
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
