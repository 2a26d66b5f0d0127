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
// Maxima of N groups that 16 lanes hold, 8 values a lane, each.  The lanes share the groups out: 5
// exchanges instead of 16 for four groups, and one lane for each quotient of a group.  A lane's
// result is that of group my_group<N>() of them; its first lane in the half warp is 16 / N times that.
template <int N> __device__ __forceinline__ int my_group() {
  const int l = threadIdx.x;
  return N == 4 ? (l >> 2) & 3 : N == 2 ? (l >> 3) & 1 : 0;
}
template <int N> __device__ __forceinline__ uint32_t group_maxima(const uint32_t (&m)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  const auto from = [](uint32_t v, int lanes) { return __shfl_xor_sync(0xffffffffu, v, lanes); };
  const bool up = threadIdx.x & 8, odd = threadIdx.x & 4;
  uint32_t r;
  if constexpr (N == 4) {
    const uint32_t even_group = max(up ? m[2] : m[0], from(up ? m[0] : m[2], 8));
    const uint32_t odd_group = max(up ? m[3] : m[1], from(up ? m[1] : m[3], 8));
    r = max(odd ? odd_group : even_group, from(odd ? even_group : odd_group, 4));
  } else {
    r = N == 2 ? max(up ? m[N - 1] : m[0], from(up ? m[0] : m[N - 1], 8)) : max(m[0], from(m[0], 8));
    r = max(r, from(r, 4));
  }
  r = max(r, from(r, 2));
  return max(r, from(r, 1));
}
// What the lanes of a half warp hold for their k-th group of N.
template <int N> __device__ __forceinline__ uint32_t of_group(uint32_t v, int k) {
  return N == 1 ? v : __shfl_sync(0xffffffffu, v, (threadIdx.x & 16) + k * (16 / N));
}
template <int N> __device__ __forceinline__ bool first_of_group() { return (threadIdx.x & (16 / N - 1)) == 0; }
// packed fp32 pairs (one instruction for two values)
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
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
// once so that their loads are in flight together and one lane takes the quotients of one row's
// group.  Bound by HBM, (2 or 4) + 1 bytes per value, and behind it by instructions in bf16: 8320 x
// 8192 35 us (5.8 TB/s; 39 with each row's maximum by itself, 44 with two rows a warp), in fp32 56 us
// (6.1 TB/s; eight rows a warp 62); 535 x 4096 2.6 us.
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
  uint32_t m[QR_UNROLL];
#pragma unroll
  for (int u = 0; u < QR_UNROLL; ++u) m[u] = v[u].amax();
  const float a = fp8_amax_floor(group_maxima<QR_UNROLL>(m));
  const uint32_t inv = __float_as_uint(FP8_MAX / a);
  const long long mine = row0 + my_group<QR_UNROLL>();
  if (first_of_group<QR_UNROLL>() && (col & ~127) < cols && mine < rows)
    scales[static_cast<long long>(col >> 7) * lds + mine] = a / FP8_MAX;
#pragma unroll
  for (int u = 0; u < QR_UNROLL; ++u) {
    float f[8];
    v[u].get(f);
    const uint2 q = fp8_codes8(f, __uint_as_float(of_group<QR_UNROLL>(inv, u)));
    if (in && row0 + u < rows) *reinterpret_cast<uint2*>(codes + (row0 + u) * ldc + col) = q;
  }
}

// ----------------------------------------------------------------------------- weight blocks
// One CTA per 128 x 128 block, held in registers between the maximum and the codes (one read):
// a half warp per row segment of 128 channels, 8 rows per thread, kept as they lie in memory.
// Bound by HBM: 20480 x 7168 in bf16 63 us (7.0 TB/s), in fp32 102 us (7.2 TB/s).
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
// Bound by HBM for large matrices with a residual (8320 x 8192 in bf16: 70 .. 72 us, 6.7 TB/s; 8320 x 7168
// with an fp32 residual 95 us, 6.9 TB/s), by instructions without (8000 x 8192: 38 us, 5.2 TB/s,
// hence the packed pairs and shared maxima), by a row's latency for few rows (one row 2.0 us).  A
// stream of bulk copies into shared memory ahead of the sums was no faster.  The test of the mean's
// range costs 1 to 2 percent, 4 to 7 where a row is a warp's (8320 x 512 4.5 -> 4.8 us).

// Sum over the block.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0.f);
}

// Sum of the squares of the values in f over the row (a warp's or the CTA's).
template <int CH, bool WARP> __device__ __forceinline__ float sum_of_squares(const float (&f)[CH][8], float* red) {
  uint64_t ss2 = 0;
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int j = 0; j < 8; j += 2) asm("fma.rn.f32x2 %0, %1, %1, %0;" : "+l"(ss2) : "l"(pair(f[k][j], f[k][j + 1])));
  float even, odd;
  unpair(ss2, even, odd);
  return WARP ? warp_sum(even + odd) : block_sum(even + odd, red);
}

// The mean of squares, with eps, of a row (in f) where it came out beyond 2^100 or below 2^-100, so that
// the sum may have overflowed or gone under: again for the row times 2^-80 (its largest magnitude is
// then between 2^-30 and 2^48) or 2^100 (2^-49 .. 2^58), which the norm takes out again.  f keeps that
// row.
template <int CH, bool WARP>
__device__ __forceinline__ float rescaled_mean(float (&f)[CH][8], float mean, float eps, int d, float* red) {
  const float s = mean > 1.0f ? 0x1p-80f : 0x1p100f;
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) f[k][j] *= s;
  if (!WARP) __syncthreads();  // (the sums in red have been read)
  return sum_of_squares<CH, WARP>(f, red) / static_cast<float>(d) + eps * s * s;
}

// Codes and scales of the row h (in f), given 1 / rms.
template <typename TX, int CH>
__device__ __forceinline__ void norm_codes(float (&f)[CH][8], float inv_rms, const TX* __restrict__ weight, int d,
                                           int t, int T, long long row, uint8_t* __restrict__ codes, long long ldc,
                                           float* __restrict__ scales, long long lds) {
  uint32_t m[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (t + k * T) * 8;
    if (weight && c < d) {
      float w[8];
      load8(weight + c, w);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint64_t u = pair(f[k][j], f[k][j + 1]);
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(u) : "l"(pair(w[j], w[j + 1])));
        unpair(u, f[k][j], f[k][j + 1]);
      }
    }
    m[k] = amax_bits8(f[k]);
  }
  // y = u * inv_rms with u = h * w, so y * (448 / max|y|) = u * (448 / max|u|): the codes do not
  // see the norm's rounding (two roundings instead of four), only the scale does.  Where 448 /
  // max|u| could overflow, or the scale's floor applies, the codes come from y itself (the factor's
  // sign says so).  Each lane does this for one of its half warp's groups.
  const float au = __uint_as_float(group_maxima<CH>(m));
  const float a = fp8_amax_floor(abs_bits(au * inv_rms));
  const bool direct = au > 0x1p-100f && a > FP8_AMAX_MIN;
  const uint32_t factor = __float_as_uint(FP8_MAX / (direct ? au : a)) | (direct ? 0u : 0x80000000u);
  const int group = (t + my_group<CH>() * T) >> 4;
  if (first_of_group<CH>() && group * 128 < d) scales[static_cast<long long>(group) * lds + row] = a / FP8_MAX;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (t + k * T) * 8;
    const uint32_t mine = of_group<CH>(factor, k);
    if (mine >> 31) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[k][j] *= inv_rms;
    }
    if (c < d) *reinterpret_cast<uint2*>(codes + row * ldc + c) = fp8_codes8(f[k], __uint_as_float(mine & 0x7fffffffu));
  }
}

// WARP: a row is a warp's, eight rows a CTA; else a CTA's.  (Two pieces a thread, all in bf16: 40 registers
// let three CTAs of 512 threads share an SM.)
template <typename TX, typename TR, bool RES, int CH, bool WARP>
__global__ void __launch_bounds__(CH == 2 && !WARP ? 512 : 1024, CH == 2 && !WARP && sizeof(TX) + sizeof(TR) == 4 ? 3 : 1)
    add_rmsnorm_fp8_kernel(const TX* __restrict__ x, long long ldx,
                           const void* residual, void* residual_out, long long ldr,
                           const TX* __restrict__ weight, int rows, int d, float eps,
                           uint8_t* __restrict__ codes, long long ldc,
                           float* __restrict__ scales, long long lds) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[32];
  const TR* res = static_cast<const TR*>(residual);
  TR* res_out = static_cast<TR*>(residual_out);
  const long long row = WARP ? static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x;
  const int t = WARP ? threadIdx.x & 31 : threadIdx.x, T = WARP ? 32 : blockDim.x;
  if (WARP && row >= rows) return;
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
  uint64_t ss2 = 0;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = (t + k * T) * 8;
    float r[8];
    px[k].get(f[k]);
    pr[k].get(r);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint64_t h = pair(f[k][j], f[k][j + 1]);
      if (RES) asm("add.rn.f32x2 %0, %0, %1;" : "+l"(h) : "l"(pair(r[j], r[j + 1])));
      asm("fma.rn.f32x2 %0, %1, %1, %0;" : "+l"(ss2) : "l"(h));
      unpair(h, f[k][j], f[k][j + 1]);
    }
    if (RES && res_out && c < d) store8(res_out + row * ldr + c, f[k]);
  }
  float even, odd;
  unpair(ss2, even, odd);
  const float sum = WARP ? warp_sum(even + odd) : block_sum(even + odd, red);
  float mean = sum / static_cast<float>(d) + eps;
  if (mean < 0x1p-100f || mean > 0x1p100f) mean = rescaled_mean<CH, WARP>(f, mean, eps, d, red);  // (uniform in the row)
  const float inv_rms = 1.0f / sqrtf(mean);
  norm_codes<TX, CH>(f, inv_rms, weight, d, t, T, row, codes, ldc, scales, lds);
}

template <typename TX, typename TR>
cudaError_t launch_norm(const void* x, long long ldx, const void* res, void* res_out, long long ldr, const void* weight,
                        int rows, int d, float eps, void* codes, long long ldc, float* scales, long long lds,
                        cudaStream_t s) {
  const int pieces = (d + 7) / 8;
  auto one = [&](auto kernel, int ch) {  // ch 0: a row is a warp's
    const int threads = ch ? ((pieces + ch - 1) / ch + 31) / 32 * 32 : 256;
    return launch_chain(kernel, dim3(ch ? rows : (rows + 7) / 8), dim3(threads), 0, s, static_cast<const TX*>(x), ldx,
                        res, res_out, ldr, static_cast<const TX*>(weight), rows, d, eps, static_cast<uint8_t*>(codes), ldc,
                        scales, lds);
  };
  // A row per warp up to 512 channels, and for many rows without a residual up to 1024: no barrier, an
  // eighth of the CTAs (8320 x 256 bf16 4.7 us, a CTA a row 9.2; 8320 x 512 7.3 / 9.3; 4000 x 768
  // without a residual 3.2 / 4.9; with fp32 residuals 4000 x 768 9.5 / 8.1, hence not).
  if (pieces <= 64 && res)
    return pieces <= 32 ? one(add_rmsnorm_fp8_kernel<TX, TR, true, 1, true>, 0) : one(add_rmsnorm_fp8_kernel<TX, TR, true, 2, true>, 0);
  if (pieces <= 64)
    return pieces <= 32 ? one(add_rmsnorm_fp8_kernel<TX, TX, false, 1, true>, 0) : one(add_rmsnorm_fp8_kernel<TX, TX, false, 2, true>, 0);
  if (pieces <= 128 && !res && rows >= 1024) return one(add_rmsnorm_fp8_kernel<TX, TX, false, 4, true>, 0);
  // Pieces per thread.  One while the GPU holds all pieces at once (152 SMs x 2048 threads), the
  // shortest way through a row: 1 x 4096 2.1 us (four 3.2), 535 x 4096 with a residual 6.0 (two 6.3).
  // Then two with a residual up to 8192 channels (8320 x 4096 39.7 us, one 45.4; 8320 x 8192 73, one
  // 94, four 74; 1357 x 7168 with an fp32 residual 18.7, one 19.6, four 19.3) and four for longer rows
  // (8320 x 16384 140, two 184) and without a residual (8320 x 4096 22.7, one 33; 8000 x 8192 41, two 51).
  const bool one_piece = pieces <= 1024 && static_cast<long long>(rows) * pieces <= 152 * 2048;
  if (!res) return one_piece ? one(add_rmsnorm_fp8_kernel<TX, TX, false, 1, false>, 1) : one(add_rmsnorm_fp8_kernel<TX, TX, false, 4, false>, 4);
  if (one_piece) return one(add_rmsnorm_fp8_kernel<TX, TR, true, 1, false>, 1);
  return pieces <= 1024 ? one(add_rmsnorm_fp8_kernel<TX, TR, true, 2, false>, 2) : one(add_rmsnorm_fp8_kernel<TX, TR, true, 4, false>, 4);
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
