// A KV cache in 4 bits (layout and arithmetic: kvq.cuh): rows quantised as they are written, and read back
// with their keys turned to new positions.
//
// Both kernels give four channels to a lane, so that a group of 32 channels is 8 lanes (its extremes three
// shuffles) and a row of one head is a warp (128 channels) or half of one (64).
#include "internal.h"
#include "kvq.cuh"

namespace cb {

namespace {

constexpr int KVQ_WARPS = 8;

__device__ __forceinline__ void load4(const bf16* p, float* f) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(u.x << 16);
  f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16);
  f[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float* f) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  f[0] = u.x;
  f[1] = u.y;
  f[2] = u.z;
  f[3] = u.w;
}
__device__ __forceinline__ void store4(bf16* p, const float* f) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
__device__ __forceinline__ void store4(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// Codes (nibbles 0 to 3) of a lane's four channels, and its group's scale and zero packed as bf16.
__device__ __forceinline__ uint32_t encode4(const float* x, uint32_t& params) {
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i] != x[i] ? INFINITY : x[i]);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float2 p = kvq_params(lo, hi);
  params = (__float_as_uint(p.x) >> 16) | (__float_as_uint(p.y) & 0xffff0000u);
  if (!(p.x < INFINITY)) return 0;
  const float inv = __frcp_rn(p.x);
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c |= kvq_code(x[i], p.x, inv, p.y) << (4 * i);
  return c;
}

template <typename T, int DH>
__global__ void __launch_bounds__(KVQ_WARPS * 32) kvq_write_kernel(KvqView c, const T* __restrict__ k, long long ldk,
                                                                   const T* __restrict__ v, long long ldv,
                                                                   const int32_t* __restrict__ seqs,
                                                                   const int32_t* __restrict__ poss, int rows,
                                                                   int32_t* status) {
  pdl_trigger();
  pdl_wait();
  constexpr int LANES = DH / 4, NG = DH / 32;
  const int L = threadIdx.x % LANES;
  const long long item = (static_cast<long long>(blockIdx.x) * KVQ_WARPS * 32 + threadIdx.x) / LANES;
  const int row = static_cast<int>(item / c.n_kv_heads), head = static_cast<int>(item % c.n_kv_heads);
  // (the lanes of a row that is left out keep up with the shuffles)
  const bool in = row < rows;
  const int pos = in ? poss[row] : -1, seq = in ? (seqs ? seqs[row] : row) : -1;
  float kx[4] = {}, vx[4] = {};
  uint8_t* blk = nullptr;
  if (pos >= 0 && seq >= 0) {
    load4(k + row * ldk + head * DH + 4 * L, kx);
    load4(v + row * ldv + head * DH + 4 * L, vx);
    blk = kvq_block(c, seq, pos, DH, status);
  }
  uint32_t kp, vp;
  const uint32_t kc = encode4(kx, kp), vc = encode4(vx, vp);
  // the value channels 8 up or down are two lanes away; a lane of the lower channels writes the first two
  // bytes of the pair's four, one of the upper the others
  const uint32_t other = __shfl_xor_sync(0xffffffffu, vc, 2);
  if (!blk) return;
  blk += static_cast<size_t>(head) * (c.page_tokens / KVQ_BLOCK) * kvq_block_bytes(DH);
  const int r = pos % KVQ_BLOCK;
  const int g = L / 8, tq = L % 8 / 2;
  *reinterpret_cast<uint16_t*>(blk + r * (DH / 2) + (tq * NG + g) * 4 + (L & 1) * 2) = static_cast<uint16_t>(kc);
  const bool upper = L & 2;
  const uint32_t lo = upper ? other : vc, hi = upper ? vc : other;
  const int n0 = 4 * (L & 1) + (upper ? 2 : 0);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int sh = 4 * ((n0 & 3) + i);
    blk[kvq_value_byte(DH, r, L / 4, n0 + i)] = static_cast<uint8_t>(((lo >> sh) & 15u) | (((hi >> sh) & 15u) << 4));
  }
  if (L % 8 == 0) {
    uint16_t* p = reinterpret_cast<uint16_t*>(blk + 16 * DH + 4 * NG * r);
    p[g] = static_cast<uint16_t>(kp);
    p[NG + g] = static_cast<uint16_t>(kp >> 16);
    p += 32 * NG;
    p[g] = static_cast<uint16_t>(vp);
    p[NG + g] = static_cast<uint16_t>(vp >> 16);
  }
}

struct KvqTurn {
  float2 cs[64];  // (cos, sin) of channel pairs i, i + head_dim / 2
};

template <typename T, int DH>
__global__ void __launch_bounds__(KVQ_WARPS * 32) kvq_read_kernel(KvqView c, const int32_t* __restrict__ seqs,
                                                                  const int32_t* __restrict__ poss, int rows,
                                                                  const __grid_constant__ KvqTurn turn, bool turned,
                                                                  T* __restrict__ k, long long ldk, T* __restrict__ v,
                                                                  long long ldv, int32_t* status) {
  pdl_trigger();
  pdl_wait();
  constexpr int LANES = DH / 4, NG = DH / 32;
  const int L = threadIdx.x % LANES;
  const long long item = (static_cast<long long>(blockIdx.x) * KVQ_WARPS * 32 + threadIdx.x) / LANES;
  const int row = static_cast<int>(item / c.n_kv_heads), head = static_cast<int>(item % c.n_kv_heads);
  const bool in = row < rows;
  const int pos = in ? poss[row] : -1, seq = in ? (seqs ? seqs[row] : row) : -1;
  const uint8_t* blk = pos >= 0 && seq >= 0 ? kvq_block(c, seq, pos, DH, status) : nullptr;
  float kx[4] = {}, vx[4] = {};
  if (blk) {
    blk += static_cast<size_t>(head) * (c.page_tokens / KVQ_BLOCK) * kvq_block_bytes(DH);
    const int r = pos % KVQ_BLOCK, g = L / 8, tq = L % 8 / 2;
    const uint32_t kc = *reinterpret_cast<const uint16_t*>(blk + r * (DH / 2) + (tq * NG + g) * 4 + (L & 1) * 2);
    const uint16_t* p = reinterpret_cast<const uint16_t*>(blk + 16 * DH + 4 * NG * r);
    const float ks = __uint_as_float(static_cast<uint32_t>(p[g]) << 16), kz = __uint_as_float(static_cast<uint32_t>(p[NG + g]) << 16);
    p += 32 * NG;
    const float vs = __uint_as_float(static_cast<uint32_t>(p[g]) << 16), vz = __uint_as_float(static_cast<uint32_t>(p[NG + g]) << 16);
    const int n0 = 4 * (L & 1), up = L & 2 ? 4 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kx[i] = ks * (static_cast<float>((kc >> (4 * i)) & 15u) + kz);
      vx[i] = vs * (static_cast<float>((blk[kvq_value_byte(DH, r, L / 4, n0 + i)] >> up) & 15) + vz);
    }
  }
  if (turned) {
    const bool second = L >= LANES / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 cs = turn.cs[4 * (second ? L - LANES / 2 : L) + i];
      const float y = __shfl_xor_sync(0xffffffffu, kx[i], LANES / 2);
      kx[i] = second ? fmaf(y, cs.y, kx[i] * cs.x) : fmaf(-y, cs.y, kx[i] * cs.x);
    }
  }
  if (!in) return;
  store4(k + row * ldk + head * DH + 4 * L, kx);
  store4(v + row * ldv + head * DH + 4 * L, vx);
}

unsigned kvq_grid(int rows, int heads, int dh) {
  const long long lanes = static_cast<long long>(rows) * heads * (dh / 4);
  return static_cast<unsigned>((lanes + KVQ_WARPS * 32 - 1) / (KVQ_WARPS * 32));
}

}  // namespace

cudaError_t launch_kvq_write(const KvqView& c, int head_dim, const void* k, long long ldk, const void* v, long long ldv,
                             cb_dtype dt, const int32_t* seq, const int32_t* pos, int rows, int32_t* status,
                             cudaStream_t s) {
  const dim3 grid(kvq_grid(rows, c.n_kv_heads, head_dim)), block(KVQ_WARPS * 32);
  auto go = [&](auto* kernel, auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_chain(kernel, grid, block, 0, s, c, static_cast<T*>(k), ldk, static_cast<T*>(v), ldv, seq, pos, rows,
                        status);
  };
  const bf16* b = nullptr;
  const float* f = nullptr;
  if (dt == CB_BF16) return head_dim == 128 ? go(kvq_write_kernel<bf16, 128>, b) : go(kvq_write_kernel<bf16, 64>, b);
  return head_dim == 128 ? go(kvq_write_kernel<float, 128>, f) : go(kvq_write_kernel<float, 64>, f);
}

cudaError_t launch_kvq_read(const KvqView& c, int head_dim, const int32_t* seq, const int32_t* pos, int rows,
                            const float* cs_host, cb_dtype dt, void* k, long long ldk, void* v, long long ldv,
                            int32_t* status, cudaStream_t s) {
  const dim3 grid(kvq_grid(rows, c.n_kv_heads, head_dim)), block(KVQ_WARPS * 32);
  KvqTurn turn = {};
  if (cs_host)
    for (int i = 0; i < head_dim / 2; ++i) turn.cs[i] = make_float2(cs_host[2 * i], cs_host[2 * i + 1]);
  auto go = [&](auto* kernel, auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_chain(kernel, grid, block, 0, s, c, seq, pos, rows, turn, cs_host != nullptr, static_cast<T*>(k), ldk,
                        static_cast<T*>(v), ldv, status);
  };
  bf16* b = nullptr;
  float* f = nullptr;
  if (dt == CB_BF16) return head_dim == 128 ? go(kvq_read_kernel<bf16, 128>, b) : go(kvq_read_kernel<bf16, 64>, b);
  return head_dim == 128 ? go(kvq_read_kernel<float, 128>, f) : go(kvq_read_kernel<float, 64>, f);
}

}  // namespace cb
