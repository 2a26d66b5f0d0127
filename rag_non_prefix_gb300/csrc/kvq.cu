// A KV cache in 4 bits (layout and arithmetic: kvq.cuh): rows quantised as they are written, and read back
// with their keys turned to new positions.
//
// Bounds: a number is 2 or 4 bytes and 5 bits, and takes some 28 instructions to write and 13 to read.  Prompts are bound by these
// and by the latency of the loads that 32 warps an SM cover (8320 rows of 8 heads of 128 written from bf16 and read back to
// fp32: 36.5 us for 124 MB, half the rate of a copy; 4096 rows of 32 heads read to bf16: 25.3 us, 3.5 TB/s; with the registers of
// 24 warps an SM 28.4); decoded tokens by one warp's chain (16 rows of 8 heads written and read back: 4.6 us, two launches).
//
// Both kernels give eight channels to a lane: a row of one head is 16 lanes (128 channels) or 8, a group of 32
// channels four of them (its extremes two shuffles), and the row's key codes are one word a lane.  A word of value codes
// belongs to four tokens (2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9 of a block), so a warp takes those four rows of
// 16 at a time: where they are such a word's tokens (a prompt from a multiple of 16 on) it moves whole words,
// else (decoded tokens, scattered ones) a token's bytes alone.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "kvq.cuh"

namespace cb {

namespace {

constexpr int KVQ_WARPS = 2;  // of a CTA (8: decoded tokens written and read back 5.0 us instead of 4.6, the other sizes alike)

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// The rows of a warp and where they lie (64 channels: eight lanes of each half of a warp).
// STEPS 2: in step k the first half takes row 2 tq + 8 k of 16, the second row 2 tq + 1 + 8 k.
// STEPS 1: two rows of the call, as they come (few rows, whose time is that of one warp's steps).
template <int DH, int STEPS> struct KvqRows {
  static constexpr int LANES = DH / 8;
  int L, tq, g;          // lane of its row; of the row's word of keys: pair of columns and group
  int row[STEPS], r[STEPS];  // this lane's rows, and which tokens of their blocks they are
  uint8_t* blk[STEPS];   // their blocks (head 0), or nullptr
  bool whole;            // the warp's four rows share their words of value codes

  // `unit`: four rows of 16 (STEPS 2), or two rows
  __device__ __forceinline__ KvqRows(const KvqView& c, const int32_t* seqs, const int32_t* poss, int rows, int unit,
                                     int32_t* status) {
    const int lane = threadIdx.x & 31, second = lane / 16;
    L = lane % LANES;
    tq = L & 3;
    g = L >> 2;
    const int quad = unit & 3;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      row[k] = STEPS == 2 ? (unit >> 2) * 16 + 2 * quad + second + 8 * k : 2 * unit + second;
      const bool in = row[k] < rows && lane % 16 < LANES;
      const int pos = in ? poss[row[k]] : -1, seq = in ? (seqs ? seqs[row[k]] : row[k]) : -1;
      blk[k] = pos >= 0 && seq >= 0 ? kvq_block(c, seq, pos, DH, status) : nullptr;
      r[k] = pos & 15;
    }
    whole = false;
    if (STEPS == 1) return;
    const uint8_t* same = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(blk[0]), 0));
    const bool mine = lane % 16 >= LANES ||
                      (same && blk[0] == same && blk[STEPS - 1] == same && r[0] == 2 * quad + second && r[STEPS - 1] == r[0] + 8);
    whole = __all_sync(0xffffffffu, mine);
  }
};

// A lane's eight numbers of a row as they are loaded (zeros where there is no row), and the smallest and largest of the four
// lanes' of a group; if a number is not finite, neither is one of these, or their difference.
struct Eight_bf16 {
  uint4 u = {};
  __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void floats(float* x) const { load8(reinterpret_cast<const bf16*>(&u), x); }
  __device__ __forceinline__ void extremes(float& lo, float& hi) const {
    // pairs throughout; at last the smallest in the lower half, the largest's negative in the upper
    auto h = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    auto bits = [](__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); };
    const uint32_t l = bits(__hmin2_nan(__hmin2_nan(h(u.x), h(u.y)), __hmin2_nan(h(u.z), h(u.w))));
    const uint32_t m = bits(__hmax2_nan(__hmax2_nan(h(u.x), h(u.y)), __hmax2_nan(h(u.z), h(u.w)))) ^ 0x80008000u;
    uint32_t both = bits(__hmin2_nan(h(__byte_perm(l, m, 0x5410)), h(__byte_perm(l, m, 0x7632))));
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) both = bits(__hmin2_nan(h(both), h(__shfl_xor_sync(0xffffffffu, both, o))));
    lo = __uint_as_float(both << 16);
    hi = -__uint_as_float(both & 0xffff0000u);
  }
};
struct Eight_f32 {
  float x[8] = {};
  __device__ __forceinline__ void load(const float* p) { load8(p, x); }
  __device__ __forceinline__ void floats(float* y) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
  }
  __device__ __forceinline__ void extremes(float& lo, float& hi) const {
    lo = hi = x[0];
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      odd = fmaf(x[i], 0.f, odd);  // NaN once a number is not finite
    }
    hi = odd == 0.f ? hi : INFINITY;
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  }
};
template <typename T> using Eight = std::conditional_t<std::is_same<T, bf16>::value, Eight_bf16, Eight_f32>;

// Codes of a lane's eight channels under their group's scale and zero (kvq_params).
template <typename E> __device__ __forceinline__ uint32_t encode8(const E& e, uint32_t params) {
  float x[8];
  e.floats(x);
  const float scale = __uint_as_float(params << 16), zero = __uint_as_float(params & 0xffff0000u);
  const uint32_t c = kvq_codes(x, scale, zero, kvq_reciprocal(scale));
  return scale < INFINITY ? c : 0;
}

template <typename T, int DH, int STEPS>
__global__ void __launch_bounds__(KVQ_WARPS * 32, 32 / KVQ_WARPS) kvq_write_kernel(KvqView c, const T* __restrict__ k, long long ldk,
                                                                   const T* __restrict__ v, long long ldv,
                                                                   const int32_t* __restrict__ seqs,
                                                                   const int32_t* __restrict__ poss, int rows, int units,
                                                                   int heads_each, int32_t* status) {
  pdl_trigger();
  pdl_wait();
  constexpr int LANES = DH / 8, NG = DH / 32;
  const int lane = threadIdx.x & 31, unit = blockIdx.x * KVQ_WARPS + (threadIdx.x >> 5);
  if (unit >= units) return;
  const KvqRows<DH, STEPS> at(c, seqs, poss, rows, unit, status);
  const int L = at.L;
  const size_t head_bytes = static_cast<size_t>(c.page_tokens / KVQ_BLOCK) * kvq_block_bytes(DH);
  const int h0 = blockIdx.y * heads_each, h1 = min(h0 + heads_each, c.n_kv_heads);
  const int mine = at.tq % (2 * STEPS);  // this lane's scale and zero: of step mine / 2, keys or values
  uint8_t* own_blk = at.tq < 2 * STEPS ? at.blk[mine / 2 && STEPS == 2 ? STEPS - 1 : 0] : nullptr;
  uint16_t* own_params = own_blk ? reinterpret_cast<uint16_t*>(own_blk + 16 * DH + 4 * NG * at.r[mine / 2 && STEPS == 2 ? STEPS - 1 : 0]) +
                                       at.g + (mine & 1) * 32 * NG : nullptr;
  for (int head = h0; head < h1; ++head) {
    uint32_t half[STEPS];  // value bytes of channels n (low nibbles) and n + 8 (high): n = 0..3 by even lanes, 4..7 by odd ones
    Eight<T> kx[STEPS], vx[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (at.blk[s]) {
        kx[s].load(k + at.row[s] * ldk + head * DH + 8 * L);
        vx[s].load(v + at.row[s] * ldv + head * DH + 8 * L);
      }
    }
    // the group's scales and zeros, of keys and values of each step, one by each of its four lanes
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      float l, h;
      kx[s].extremes(l, h);
      if (mine == 2 * s) lo = l, hi = h;
      vx[s].extremes(l, h);
      if (mine == 2 * s + 1) lo = l, hi = h;
    }
    const uint32_t params = kvq_params(lo, hi);
    if (own_params) {
      uint16_t* p = own_params + head * (head_bytes / 2);
      p[0] = static_cast<uint16_t>(params);
      p[NG] = static_cast<uint16_t>(params >> 16);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const uint32_t kc = encode8(kx[s], __shfl_sync(0xffffffffu, params, (lane & ~3) + 2 * s));
      const uint32_t vc = encode8(vx[s], __shfl_sync(0xffffffffu, params, (lane & ~3) + 2 * s + 1));
      const uint32_t other = __shfl_xor_sync(0xffffffffu, vc, 1);
      const uint32_t lo = L & 1 ? other >> 16 : vc, hi = L & 1 ? vc >> 16 : other;
      // nibbles 0 to 3 of both, interleaved to bytes
      const uint32_t lo2 = (lo & 0xf) | (lo & 0xf0) << 4 | (lo & 0xf00) << 8 | (lo & 0xf000) << 12;
      const uint32_t hi2 = (hi & 0xf) | (hi & 0xf0) << 4 | (hi & 0xf00) << 8 | (hi & 0xf000) << 12;
      half[s] = lo2 | hi2 << 4;
      if (!at.blk[s]) continue;
      uint8_t* blk = at.blk[s] + head * head_bytes;
      const int r = at.r[s];
      *reinterpret_cast<uint32_t*>(blk + r * (DH / 2) + (at.tq * NG + at.g) * 4) = kc;
      if (!at.whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          blk[kvq_value_byte(DH, r, L >> 1, 4 * (L & 1) + i)] = static_cast<uint8_t>(half[s] >> (8 * i));
      }
    }
    if (STEPS == 2 && at.whole) {
      // a lane has the bytes of tokens 2 tq and 2 tq + 8, the lane 16 away those of 2 tq + 1 and 2 tq + 9: two of
      // the four words each
      const bool second = lane >= 16;
      const uint32_t pair0 = __byte_perm(half[0], half[STEPS - 1], 0x5140), pair1 = __byte_perm(half[0], half[STEPS - 1], 0x7362);  // n 0, 1; n 2, 3
      const uint32_t got = __shfl_xor_sync(0xffffffffu, second ? pair0 : pair1, 16);
      const uint32_t w0 = second ? __byte_perm(got, pair1, 0x5410) : __byte_perm(pair0, got, 0x5410);
      const uint32_t w1 = second ? __byte_perm(got, pair1, 0x7632) : __byte_perm(pair0, got, 0x7632);
      if (lane % 16 < LANES) {
        uint8_t* blk = at.blk[0] + head * head_bytes;
        const int at0 = kvq_value_byte(DH, at.r[0] & ~9, L >> 1, 4 * (L & 1) + (second ? 2 : 0));
        *reinterpret_cast<uint32_t*>(blk + at0) = w0;
        *reinterpret_cast<uint32_t*>(blk + at0 + 64) = w1;
      }
    }
  }
}

// `wide`: rows start at multiples of 32 bytes, and eight fp32 numbers are one store
__device__ __forceinline__ void store_row(bf16* p, const float* x, bool) { store8(p, x); }
__device__ __forceinline__ void store_row(float* p, const float* x, bool wide) {
  if (wide)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
                 "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
  else
    store8(p, x);
}

struct KvqTurn {
  float2 cs[64];  // (cos, sin) of channel pairs i, i + head_dim / 2
};

template <typename T, int DH, int STEPS>
__global__ void __launch_bounds__(KVQ_WARPS * 32, 32 / KVQ_WARPS) kvq_read_kernel(KvqView c, const int32_t* __restrict__ seqs,
                                                                  const int32_t* __restrict__ poss, int rows, int units,
                                                                  int heads_each, const __grid_constant__ KvqTurn turn,
                                                                  bool turned, bool wide, T* __restrict__ k, long long ldk,
                                                                  T* __restrict__ v, long long ldv, int32_t* status) {
  __shared__ float2 cs[64];
  // (read one by one: an indexed kernel argument is fetched lane after lane)
  if (turned)
    for (int i = threadIdx.x; i < DH / 2; i += KVQ_WARPS * 32) cs[i] = turn.cs[i];
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  constexpr int LANES = DH / 8, NG = DH / 32;
  const int lane = threadIdx.x & 31, unit = blockIdx.x * KVQ_WARPS + (threadIdx.x >> 5);
  if (unit >= units) return;
  const KvqRows<DH, STEPS> at(c, seqs, poss, rows, unit, status);
  const int L = at.L;
  const bool upper = L >= LANES / 2;
  float co[8], si[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = turned ? cs[(8 * L + i) % (DH / 2)] : make_float2(1.f, 0.f);
    co[i] = x.x;
    si[i] = upper ? x.y : -x.y;
  }
  const size_t head_bytes = static_cast<size_t>(c.page_tokens / KVQ_BLOCK) * kvq_block_bytes(DH);
  const int h0 = blockIdx.y * heads_each, h1 = min(h0 + heads_each, c.n_kv_heads);
  // WHOLE: the warp's four rows share their words; every load is on its way before the first is needed
  auto heads = [&](auto whole_rows) {
    constexpr bool WHOLE = decltype(whole_rows)::value;
    for (int head = h0; head < h1; ++head) {
      uint32_t kc[STEPS] = {}, vc[WHOLE ? 1 : STEPS][8] = {};
      uint16_t prm[STEPS][4] = {};  // scale and zero of the key, of the value
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        if (!at.blk[s]) continue;
        const uint8_t* blk = at.blk[s] + head * head_bytes;
        const int r = at.r[s];
        kc[s] = *reinterpret_cast<const uint32_t*>(blk + r * (DH / 2) + (at.tq * NG + at.g) * 4);
        const uint16_t* p = reinterpret_cast<const uint16_t*>(blk + 16 * DH + 4 * NG * r) + at.g;
#pragma unroll
        for (int i = 0; i < 4; ++i) prm[s][i] = p[(i & 1) * NG + (i >> 1) * 32 * NG];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!WHOLE)
            vc[s][i] = blk[kvq_value_byte(DH, r, L >> 1, i)];
          else if (s == 0)
            vc[0][i] = *reinterpret_cast<const uint32_t*>(blk + kvq_value_byte(DH, r & ~9, L >> 1, i));
        }
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        float kx[8], vx[8];
        const float ks = bf(prm[s][0]), kz = bf(prm[s][1]), vs = bf(prm[s][2]), vz = bf(prm[s][3]);
        const int up = (WHOLE ? 8 * (2 * (at.r[s] & 1) + (at.r[s] >> 3)) : 0) + (L & 1 ? 4 : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // code + zero (9 bits) first: scale times zero alone may pass fp32's range where the value does not
          kx[i] = (static_cast<float>((kc[s] >> (4 * i)) & 15u) + kz) * ks;  // (exact: 17 bits)
          vx[i] = (static_cast<float>((vc[WHOLE ? 0 : s][i] >> up) & 15u) + vz) * vs;
        }
        if (turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = __shfl_xor_sync(0xffffffffu, kx[i], LANES / 2);
            kx[i] = fmaf(y, si[i], kx[i] * co[i]);
          }
        }
        if (at.row[s] < rows && lane % 16 < LANES) {
          store_row(k + at.row[s] * ldk + head * DH + 8 * L, kx, wide);
          store_row(v + at.row[s] * ldv + head * DH + 8 * L, vx, wide);
        }
      }
    }
  };
  if (STEPS == 2 && at.whole)
    heads(std::true_type());
  else
    heads(std::false_type());
}

// Units of rows, and the heads that a warp takes one after the other: a head each while there are few, more where
// that would only look up the rows again: once there are more than `want` warps (measured, 8320 rows of 8 heads written and read
// back: 36.6 us where written at 4096, 36.7 at 8192, 38.9 at 16384; 4096 rows of 32 heads read: 27.3 us at 3000, 24.7 at
// 4096, 25.7 at 8192).  One step up to 8192 rows and heads: there a warp's chain of loads and stores is the time.
struct KvqPlan {
  int steps, units, heads_each;
  dim3 grid;
};
KvqPlan kvq_plan(int rows, int heads, int want) {
  KvqPlan p;
  p.steps = static_cast<long long>(rows) * heads <= 8192 ? 1 : 2;
  p.units = p.steps == 1 ? (rows + 1) / 2 : (rows + 15) / 16 * 4;
  const long long warps = static_cast<long long>(p.units) * heads;
  p.heads_each = static_cast<int>(std::min<long long>(heads, std::max<long long>(1, warps / want)));
  p.grid = dim3((p.units + KVQ_WARPS - 1) / KVQ_WARPS, (heads + p.heads_each - 1) / p.heads_each);
  return p;
}

}  // namespace

cudaError_t launch_kvq_write(const KvqView& c, int head_dim, const void* k, long long ldk, const void* v, long long ldv,
                             cb_dtype dt, const int32_t* seq, const int32_t* pos, int rows, int32_t* status,
                             cudaStream_t s) {
  const KvqPlan plan = kvq_plan(rows, c.n_kv_heads, 8192);
  const dim3 block(KVQ_WARPS * 32);
  auto go = [&](auto* kernel, auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_chain(kernel, plan.grid, block, 0, s, c, static_cast<T*>(k), ldk, static_cast<T*>(v), ldv, seq, pos, rows,
                        plan.units, plan.heads_each, status);
  };
  const bool one = plan.steps == 1;
  const bf16* b = nullptr;
  const float* f = nullptr;
  if (dt == CB_BF16) {
    if (head_dim == 128) return one ? go(kvq_write_kernel<bf16, 128, 1>, b) : go(kvq_write_kernel<bf16, 128, 2>, b);
    return one ? go(kvq_write_kernel<bf16, 64, 1>, b) : go(kvq_write_kernel<bf16, 64, 2>, b);
  }
  if (head_dim == 128) return one ? go(kvq_write_kernel<float, 128, 1>, f) : go(kvq_write_kernel<float, 128, 2>, f);
  return one ? go(kvq_write_kernel<float, 64, 1>, f) : go(kvq_write_kernel<float, 64, 2>, f);
}

cudaError_t launch_kvq_read(const KvqView& c, int head_dim, const int32_t* seq, const int32_t* pos, int rows,
                            const float* cs_host, cb_dtype dt, void* k, long long ldk, void* v, long long ldv,
                            int32_t* status, cudaStream_t s) {
  const KvqPlan plan = kvq_plan(rows, c.n_kv_heads, 4096);
  const dim3 block(KVQ_WARPS * 32);
  KvqTurn turn = {};
  if (cs_host)
    for (int i = 0; i < head_dim / 2; ++i) turn.cs[i] = make_float2(cs_host[2 * i], cs_host[2 * i + 1]);
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0 && ldk % 8 == 0 && ldv % 8 == 0;
  auto go = [&](auto* kernel, auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_chain(kernel, plan.grid, block, 0, s, c, seq, pos, rows, plan.units, plan.heads_each, turn,
                        cs_host != nullptr, wide, static_cast<T*>(k), ldk, static_cast<T*>(v), ldv, status);
  };
  const bool one = plan.steps == 1;
  bf16* b = nullptr;
  float* f = nullptr;
  if (dt == CB_BF16) {
    if (head_dim == 128) return one ? go(kvq_read_kernel<bf16, 128, 1>, b) : go(kvq_read_kernel<bf16, 128, 2>, b);
    return one ? go(kvq_read_kernel<bf16, 64, 1>, b) : go(kvq_read_kernel<bf16, 64, 2>, b);
  }
  if (head_dim == 128) return one ? go(kvq_read_kernel<float, 128, 1>, f) : go(kvq_read_kernel<float, 128, 2>, f);
  return one ? go(kvq_read_kernel<float, 64, 1>, f) : go(kvq_read_kernel<float, 64, 2>, f);
}

}  // namespace cb
