// The 4-bit form of a KV cache (cb_kvq_*): its layout and its arithmetic, shared by the kernels
// that write, read and attend to it.
//
// A group is 32 consecutive channels of one token's key or value of one head:
//   scale = the smallest bf16 number >= max(d / 14.75, a / 64, 2^-120),  d = hi - lo, a = max(|lo|, |hi|)
//   zero  = floor(4 lo / scale) / 4,   code = clamp(nearest(x / scale - zero), 0, 15)
//   value = scale * (code + zero)
// The zero is a multiple of 1/4 of at most 64, so bf16 holds it; 14.75 steps and a zero at most 1/4 step too
// low reach over the group.  code + zero has 9 bits and scale 8: the value is exact in fp32 (infinite beyond its range;
// scale zero alone may be where the value is not, so it is not formed), and so is
// (n + 1/2 + zero) * scale, by which the nearest code is decided exactly without a division.
//
// Block of 16 tokens of one head, 20 D bytes (D channels, NG = D / 32 groups), the memory a tensor-core
// fragment is loaded from without rearrangement:
//   key codes    token r at r D / 2: word (tq NG + g) holds channels 32 g + 8 tq + i in nibble i, so the lane
//                of key row r and column pair tq finds its operands of every group in one 16-byte piece
//   value codes  at 8 D: word ((j / 4) 128 + n 16 + tq 4 + j % 4) holds channels 16 j + n (low nibbles) and
//                16 j + n + 8 (high ones) of tokens 2 tq, 2 tq + 8, 2 tq + 1, 2 tq + 9 (bytes 0 to 3): one
//                operand fragment of 16 channels x 16 tokens a word and lane, and a byte belongs to one token
//   key scales   at 16 D: token r at 4 NG r, NG bf16 scales, then NG zeros
//   value scales 64 NG bytes further, the same
#pragma once
#include "common.cuh"
#include "internal.h"

namespace cb {

constexpr int KVQ_BLOCK = 16;
__host__ __device__ constexpr int kvq_block_bytes(int dh) { return 20 * dh; }

// block of 16 tokens that holds position pos of sequence seq, head 0; nullptr (and the status bit) if there
// is none.  Blocks of the following heads are page_tokens / 16 blocks apart.
__device__ __forceinline__ uint8_t* kvq_block(const KvqView& c, int seq, int pos, int dh, int32_t* status) {
  if (seq >= c.n_seqs || pos / c.page_tokens >= c.max_pages) {
    set_status(status, ST_RANGE);
    return nullptr;
  }
  const int slot = pos / c.page_tokens;
  const int page = c.table[seq * c.ld_table + slot];
  if (page < 0 || page >= c.n_pages) {
    set_status(status, ST_RANGE);
    return nullptr;
  }
  const size_t blocks = c.page_tokens / KVQ_BLOCK;
  return c.pool + (static_cast<size_t>(page) * c.n_kv_heads * blocks + (pos - slot * c.page_tokens) / KVQ_BLOCK) *
                      kvq_block_bytes(dh);
}

// byte of value channels 16 j + n and 16 j + n + 8 of token r
__device__ __forceinline__ int kvq_value_byte(int dh, int r, int j, int n) {
  return 8 * dh + 512 * (j >> 2) + 64 * n + 16 * ((r & 7) >> 1) + 4 * (j & 3) + 2 * (r & 1) + (r >> 3);
}

__device__ __forceinline__ float bf16_up(float x) {  // the smallest bf16 number not below x >= 0
  return __uint_as_float((__float_as_uint(x) + 0xffffu) & 0xffff0000u);
}

__device__ __forceinline__ float kvq_reciprocal(float scale) {  // approximately
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  return inv;
}

// Scale (lower half) and zero (upper) of a group whose smallest and largest numbers are lo and hi, as bf16 (hi - lo not finite: NaN).
// Quotients are estimated and put right by exact products (bf16 times 14.75: 14 bits).
__device__ __forceinline__ uint32_t kvq_params(float lo, float hi) {
  const float d = __fsub_rn(hi, lo), a = fmaxf(-lo, hi);
  float s = bf16_up(fmaxf(__fmul_rn(d, 1.f / 14.75f), 7.52316385e-37f));  // (2^-120)
  const float next = __uint_as_float(__float_as_uint(s) + 0x10000u), prev = __uint_as_float(__float_as_uint(s) - 0x10000u);
  if (__fmul_rn(s, 14.75f) < d)
    s = next;
  else if (__fmul_rn(prev, 14.75f) >= d)
    s = prev;
  const float scale = fmaxf(fmaxf(s, bf16_up(a * 0.015625f)), 7.52316385e-37f);
  float zero = 0.25f * floorf(4.f * __fmul_rn(lo, kvq_reciprocal(scale)));
  if (__fmul_rn(zero, scale) > lo)
    zero -= 0.25f;
  else if (__fmul_rn(zero + 0.25f, scale) <= lo)
    zero += 0.25f;
  return d < INFINITY ? __float_as_uint(scale) >> 16 | __float_as_uint(zero) : 0x7fc07fc0u;
}

// The codes c of eight numbers, those near a tie put right (a function of its own, so that the usual way is short).
inline __device__ __noinline__ uint32_t kvq_ties(uint32_t c, float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7,
                                          float scale, float zero, float inv) {
  const float mul = inv * (1.f / 15.f), add = zero * (-1.f / 15.f);
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __saturatef(fmaf(x[i], mul, add));
    const float n = fmaf(y, 15.f, 12582912.f) - 12582912.f, f = fmaf(y, 15.f, -n);
    if (fabsf(f) > 0.4999f) {
      const float side = copysignf(1.f, f), e = side * __fmaf_rn(-(n + 0.5f * side + zero), scale, x[i]);
      if (e > 0.f || (e == 0.f && (c >> (4 * i) & 1))) c += (f > 0.f ? 1u : 0xffffffffu) << (4 * i);
    }
  }
  return c;
}

// Codes of eight numbers of a group, one a nibble: the nearest to x / scale - zero, ties to even, exactly.  The
// estimate by the reciprocal is off by less than 2^-15 of a step (|x / scale| <= 80, a few roundings), so what lies
// farther from a tie is right; near a tie n +- 1/2 (hardly ever: one look for all eight) the sign of x - (n +- 1/2 + zero) scale,
// one fused operation with an exact factor, which keeps a sign, decides.
__device__ __forceinline__ uint32_t kvq_codes(const float* x, float scale, float zero, float inv) {
  const float mul = inv * (1.f / 15.f), add = zero * (-1.f / 15.f);
  uint32_t c = 0;
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __saturatef(fmaf(x[i], mul, add));  // code / 15 in 0..1
    const float r = fmaf(y, 15.f, 12582912.f);            // (its last bits are the nearest whole number)
    far = fmaxf(far, fabsf(fmaf(y, 15.f, 12582912.f - r)));
    c += __float_as_uint(r) << (4 * i);
  }
  c -= 0x4b400000u * 0x11111111u;
  return far > 0.4999f ? kvq_ties(c, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], scale, zero, inv) : c;
}

}  // namespace cb
