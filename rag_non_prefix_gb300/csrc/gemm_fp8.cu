// Product of two e4m3 matrices with a scale per group of 128 channels of a row of A (tokens) and
// per 128 x 128 block of B (weights):
//   acc[m][n] = sum over groups g of  sa[g][m] * sb[n / 128][g] * sum_{k in g} A[m][k] B[n][k]
// The codes' products of a group are summed in fp32 before the group's two scales multiply them.
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace cb {

namespace {

__device__ __forceinline__ float e4m3_f(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}
__device__ __forceinline__ float silu(float x) { return x / (1.0f + __expf(-x)); }

// 16 tokens x 128 output features per CTA, thread t takes feature t % 128 of 8 tokens.
constexpr int TOK = 16;
template <bool SWIGLU>
__global__ void __launch_bounds__(256) gemm_fp8_simple_kernel(Fp8Gemm p) {
  pdl_trigger();
  pdl_wait();
  __shared__ float as[TOK][128];
  __shared__ uint32_t amax[TOK];
  const int t = threadIdx.x, f = t & 127, half = t >> 7;
  const int m0 = blockIdx.y * TOK, n0 = blockIdx.x * 128, n = n0 + f;
  const int width = SWIGLU ? p.N / 2 : p.N;
  float acc[SWIGLU ? 2 : 1][8] = {};
  for (int g = 0; g * 128 < p.K; ++g) {
    __syncthreads();
    for (int i = t; i < TOK * 128; i += 256) {
      const int m = m0 + i / 128, k = g * 128 + i % 128;
      as[i / 128][i % 128] = m < p.M && k < p.K ? e4m3_f(p.a[static_cast<long long>(m) * p.lda + k]) : 0.f;
    }
    __syncthreads();
    if (n >= width) continue;
    const int nk = min(128, p.K - g * 128);
#pragma unroll
    for (int w = 0; w < (SWIGLU ? 2 : 1); ++w) {
      const uint8_t* b = (w ? p.b2 : p.b) + static_cast<long long>(n) * (w ? p.ldb2 : p.ldb) + g * 128;
      float part[8] = {};
      for (int k = 0; k < nk; ++k) {
        const float bv = e4m3_f(b[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) part[j] = fmaf(as[half * 8 + j][k], bv, part[j]);
      }
      const float sb = (w ? p.b2_scale : p.b_scale)[static_cast<long long>(n >> 7) * (w ? p.ld_b2s : p.ld_bs) + g];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int m = m0 + half * 8 + j;
        if (m < p.M) acc[w][j] = fmaf(part[j], p.a_scale[static_cast<long long>(g) * p.ld_as + m] * sb, acc[w][j]);
      }
    }
  }
  if (SWIGLU) {
    if (t < TOK) amax[t] = __float_as_uint(FP8_AMAX_MIN);
    __syncthreads();
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = silu(acc[0][j]) * acc[SWIGLU ? 1 : 0][j];
      if (n < width) atomicMax(&amax[half * 8 + j], __float_as_uint(y[j]) & 0x7fffffffu);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int m = m0 + half * 8 + j;
      if (m >= p.M || n >= width) continue;
      const float a = __uint_as_float(amax[half * 8 + j]);
      static_cast<uint8_t*>(p.c)[static_cast<long long>(m) * p.ldc + n] =
          __nv_cvt_float_to_fp8(y[j] * (FP8_MAX / a), __NV_SATFINITE, __NV_E4M3);
      if (f == 0) p.c_scale[static_cast<long long>(blockIdx.x) * p.ld_cs + m] = a / FP8_MAX;
    }
    return;
  }
  if (n >= width) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int m = m0 + half * 8 + j;
    if (m >= p.M) continue;
    const long long o = static_cast<long long>(m) * p.ldc + n;
    if (p.epilogue == CB_FP8_STORE_BF16)
      static_cast<bf16*>(p.c)[o] = __float2bfloat16_rn(acc[0][j]);
    else
      static_cast<float*>(p.c)[o] = p.epilogue == CB_FP8_ADD_F32 ? p.addend[o] + acc[0][j] : acc[0][j];
  }
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8Gemm& p, cudaStream_t s) {
  if (p.M <= 0) return cudaSuccess;
  const bool swiglu = p.epilogue == CB_FP8_SWIGLU_FP8;
  const int width = swiglu ? p.N / 2 : p.N;
  const dim3 grid((width + 127) / 128, (p.M + TOK - 1) / TOK);
  return swiglu ? launch_chain(gemm_fp8_simple_kernel<true>, grid, dim3(256), 0, s, p)
                : launch_chain(gemm_fp8_simple_kernel<false>, grid, dim3(256), 0, s, p);
}

}  // namespace cb
