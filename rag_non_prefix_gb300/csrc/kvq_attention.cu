// Attention of a few new queries per sequence over a KV cache in 4 bits (layout: kvq.cuh).
//
//   out = sum_j softmax_j(scale q . k_j) v_j,  j <= the query's position
//   q . k     = sum_g scale_g (sum_c q_c code_c + zero_g sum_c q_c)
//   sum p v_c = sum_j (p_j scale_jg) (code_jc + zero_jg)
// The codes enter the tensor core as they are, as the bf16 numbers 16 + code (two nibbles of a word become
// two operands by one shift and one logic operation), so keys and values are never rounded.  Keys: the accumulator
// starts at (zero - 16) sum_c q_c.  Values: two more products with the operands zero and -16 (both exact in bf16)
// go into the same accumulator, which so holds the true sums; kept apart, the sums of code and zero of a long
// context would be hundreds of times larger than the result, and so what the accumulator's rounding towards zero leaves of
// them.  p scale is rounded to bf16, and the same rounded number multiplies code and zero, so its rounding is one of 2^-8
// of the value itself.  fp32 outputs: queries and p scale enter as three bf16 parts each, so that nothing is
// lost, with code - 8 as the operand, the zeros' part in fp32 arithmetic, and blocks of 16 keys added in fp32 outside of
// the tensor core.
//
// mma.sync m16n8k16 and not tcgen05: 1 to 16 queries share a key, so the products are small beside the
// cache's bytes and the operands go from the cache to registers without a rearrangement.  Keys (scores) and channels (values) lie on the 16
// rows, the queries of a KV head on the 8 columns: the scores' accumulators, scaled and transposed by movmatrix, are the
// second product's operand.
//
// Work: a unit is one KV head of one tile of 8 NT query rows (a sequence's tokens x the heads of its group), cut into
// quanta of 64 keys.  All quanta stand in one row, divided evenly over the CTAs; a CTA whose share ends inside a unit
// writes its part (sums, maximum) to scratch, and whichever CTA of that unit is the last to finish
// merges the parts in the order of the keys, so results repeat exactly.  In a CTA each of 4 warps takes a block of 16
// keys of a quantum, through a ring of its own in shared memory; no warp waits for another before the end.
//
// Bounds (8 KV heads of 128): long caches by the instructions, some 1000 a pair of blocks for 5 KB, and by 7 to 10 us of units'
// beginnings, ends and merges: 32 ragged sequences of up to 8320 keys, groups of 7, 64 us, 2.7 TB/s of cache.  4 tokens of 16
// sequences, groups of 8 (two units of 16 rows a KV head, each of which reads the cache) 109 us; fp32 outputs 45 us for 4 x 4128
// keys of 32 KV heads, three products for each of the others; one sequence of 3200 keys 15 us, a chain of latencies (share 1.7,
// first loads 1.9, keys 2.6, part to memory 1.9, merge 3.3 us).  Four warps a CTA, four CTAs an SM: 128 registers a thread hold the
// loop (32 sequences: with five CTAs spills, with eight warps a CTA, which wait for each other, 69 us, with two, whose parts are
// many, 105).
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "kvq.cuh"

namespace cb {

namespace {

typedef unsigned long long u64;
constexpr int AW = 4;                    // warps per CTA
constexpr int QUANTUM = AW * KVQ_BLOCK;  // keys
// quanta of a CTA, at least, where there are few: fewer make more parts to merge (one sequence of 3200 keys: 17.0 us with 2, 15.0 with 4,
// 16.1 with 8, 21.7 with 16)
constexpr int MIN_SHARE = 4;
// what a unit costs beside its quanta (queries, first loads, merging), in quanta (32 ragged sequences and one: 83.5 and 17.7 us with 0,
// 64.9 and 17.0 with 3, 64.7 and 15.0 with 6, 65.1 and 18.1 with 9)
constexpr int UNIT_COST = 6;
constexpr int MAX_ROWS = 16;             // query rows per tile at most
constexpr float LAZY = 6.f;              // the running maximum moves once a score passes it by 2^6
constexpr float LOWEST = -3.40282347e38f;  // the maximum of no scores: finite, so that scores of -infinity have a weight of zero beside it

__host__ __device__ constexpr int slot_floats(int dh) { return MAX_ROWS * (dh + 2); }

struct KvqAttn {
  KvqView c;
  const void* q;
  long long ldq;
  const int32_t* q_pos;  // [n_seqs][T]
  int T, G;
  float scale_log2;
  void* out;
  long long ldo;
  int* counters;  // [KVQ_MAX_CTAS], zero between calls
  float* parts;   // 2 slots a CTA
  int tiles_per_seq, n_tiles;
  int32_t* status;
};

__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 + nibbles i and i + 4 of a word as two bf16 (16 is 0x4180, with 3 bits below the units); CENTRED: less 24
// (both constants in registers: one logic operation)
template <int I, bool CENTRED> __device__ __forceinline__ uint32_t nibbles(uint32_t x, uint32_t mask, uint32_t sixteen) {
  uint32_t y, r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(I == 0 ? x << 3 : x >> (4 * I - 3)), "r"(mask), "r"(sixteen));
  if (!CENTRED) return y;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x41c041c0u));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// The bf16 parts of x and y, packed: NP parts whose sum is (x, y), exactly for NP = 3; x and y become what is left.
__device__ __forceinline__ uint32_t split_off(float& x, float& y) {
  const uint32_t u = pack_bf16x2(x, y);
  x -= lo_f(u);
  y -= hi_f(u);
  return u;
}

// Quanta of a unit that sees len keys: UNIT_COST without keys first.
__device__ __forceinline__ int quanta_of(int len) { return UNIT_COST + len / QUANTUM + (len % QUANTUM != 0); }

// a / b for numbers that are hardly ever beyond 32 bits
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return a >> 32 | b >> 32 ? a / b : static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// Quanta of a unit of tile `ti`, and the number of keys that its rows see.
__device__ __forceinline__ int tile_quanta(const KvqAttn& p, int ti, int rows, int& len) {
  const int seq = ti / p.tiles_per_seq, r0 = (ti - seq * p.tiles_per_seq) * rows;
  const int t1 = (min(r0 + rows, p.T * p.G) - 1) / p.G;
  int top = -1;
  for (int t = r0 / p.G; t <= t1; ++t) top = max(top, p.q_pos[static_cast<long long>(seq) * p.T + t]);
  const int cap = p.c.max_pages * p.c.page_tokens;
  if (top >= cap) set_status(p.status, ST_RANGE);
  len = min(top, cap - 1) + 1;
  return quanta_of(len);
}

template <int DH> struct Words;  // a lane's key codes of one token: a word per group
template <> struct Words<128> { typedef uint4 type; };
template <> struct Words<64> { typedef uint2 type; };

// T: queries and outputs; NT: column tiles of 8 query rows; NP: bf16 parts of a query or weight.
template <typename T, int DH, int NT, int NP> struct Attn {
  static constexpr int NG = DH / 32, R = 8 * NT, BLK = kvq_block_bytes(DH);
  static constexpr int STAGES = 4;
  static constexpr int ROW = DH + 4;  // pitch of the merge buffer, free of bank conflicts
  static constexpr int RING = AW * STAGES * BLK;
  static constexpr int QUERIES = NT * NP * NG * 2 * 32 * 8 + NT * NG * 32 * 16;
  static constexpr int MERGE = AW * R * ROW * 4;
  static constexpr int WEIGHTS = AW * 2 * KVQ_MAX_CTAS * 4;  // a warp's (maximum or weight, sum) of a row's parts
  static constexpr int WORK = std::max(std::max(RING, MERGE), WEIGHTS);
  static constexpr int SMEM = WORK + QUERIES;

  static constexpr bool CENTRED = NP > 1;
  static constexpr float OFF = CENTRED ? 8.f : -16.f;  // what the operands' offset leaves of a zero

  int lane;
  uint32_t mask, sixteen, minus16[4];  // (an operand of four registers)
  const uint2* qb;   // this lane's query operands in shared memory: [NT][NP][NG][2] pairs (b0, b1), 32 lanes apart
  const float4* qs;  // sums of the queries' groups, of this lane's two columns, and OFF times them: [NT][NG], 32 lanes apart
  float o[NT][DH / 16][4];
  float corr[NT][NG][2];  // (fp32) this lane's keys' sums with the zeros
  float m[NT][2], l[NT][2];
  int lim[NT][2];  // last key of this lane's two columns

  // The tile's queries, a group by each warp, and the columns' last keys: first the loads (float q[NT][8], which the
  // caller keeps while it starts others), then into shared memory, with this lane's state.
  __device__ __forceinline__ void load_q(const KvqAttn& p, int seq, int r0, int head, float (&f)[NT][8]) {
    // read once: the compiler would fetch and rebuild them in every block
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
    asm volatile("mov.u32 %0, 0x00780078;" : "=r"(mask));
    asm volatile("mov.u32 %0, 0x41804180;" : "=r"(sixteen));
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("mov.u32 %0, 0xc180c180;" : "=r"(minus16[i]));
    const int rr = lane >> 2, tq = lane & 3, rows = p.T * p.G, w = threadIdx.x >> 5;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = r0 + nt * 8 + rr;
      const int t = row < rows ? row / p.G : 0, g = row - t * p.G;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[nt][i] = 0.f;
      if (row < rows && w < NG)
        load8(static_cast<const T*>(p.q) + (static_cast<long long>(seq) * p.T + t) * p.ldq +
                  static_cast<long long>(head * p.G + g) * DH + 8 * tq + 32 * w,
              f[nt]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = r0 + nt * 8 + 2 * tq + c;
        lim[nt][c] = col < rows ? p.q_pos[static_cast<long long>(seq) * p.T + col / p.G] : -1;
      }
    }
  }
  __device__ __forceinline__ void start(uint8_t* dst, float (&f)[NT][8]) {
    const int tq = lane & 3, grp = threadIdx.x >> 5;
    uint2* b = reinterpret_cast<uint2*>(dst) + lane;
    float4* sums = reinterpret_cast<float4*>(dst + NT * NP * NG * 2 * 32 * 8) + lane;
    qb = b;
    qs = sums;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (grp < NG) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += f[nt][i];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const float s0 = __shfl_sync(0xffffffffu, sum, 8 * tq), s1 = __shfl_sync(0xffffffffu, sum, 8 * tq + 4);
        sums[(nt * NG + grp) * 32] = make_float4(s0, s1, OFF * s0, OFF * s1);
#pragma unroll
        for (int np = 0; np < NP; ++np) {
          uint32_t u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = split_off(f[nt][i], f[nt][i + 4]);
          b[((nt * NP + np) * NG + grp) * 2 * 32] = make_uint2(u[0], u[1]);
          b[(((nt * NP + np) * NG + grp) * 2 + 1) * 32] = make_uint2(u[2], u[3]);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = LOWEST;
        l[nt][c] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) corr[nt][g][c] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < DH / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
    }
  }

  // the last key that every row of the tile sees (-1: a row sees none)
  __device__ __forceinline__ int seen_by_all(const KvqAttn& p, int r0) const {
    const int tq = lane & 3, rows = p.T * p.G;
    int x = 0x7fffffff;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (r0 + nt * 8 + 2 * tq + c < rows) x = min(x, lim[nt][c]);
    x = min(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return max(min(x, __shfl_xor_sync(0xffffffffu, x, 2)), -1);
  }

  // Scores (times 1 / scale) of the 16 keys of each of two blocks in shared memory: keys rr and rr + 8, columns
  // 2 tq and 2 tq + 1.
  __device__ __forceinline__ void scores(const uint8_t* blk0, const uint8_t* blk1, float (&s)[2][NT][4]) const {
    const int rr = lane >> 2, tq = lane & 3;
    uint32_t w[2][2][NG], ks[2][2][NG / 2], kz[2][2][NG / 2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* blk = u ? blk1 : blk0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        typedef typename Words<DH>::type W;
        *reinterpret_cast<W*>(w[u][h]) = *reinterpret_cast<const W*>(blk + (rr + 8 * h) * (DH / 2) + tq * 4 * NG);
        const uint32_t* prm = reinterpret_cast<const uint32_t*>(blk + 16 * DH + 4 * NG * (rr + 8 * h));
#pragma unroll
        for (int i = 0; i < NG / 2; ++i) {
          ks[u][h][i] = prm[i];
          kz[u][h][i] = prm[NG / 2 + i];
        }
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      auto half = [&](uint32_t x) { return g & 1 ? hi_f(x) : lo_f(x); };
      float c[2][NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float4 q = qs[(nt * NG + g) * 32];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) c[u][nt][i] = fmaf(half(kz[u][i >> 1][g / 2]), i & 1 ? q.y : q.x, i & 1 ? q.w : q.z);
      }
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        uint32_t a[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[u][h] = step ? nib<2>(w[u][h][g]) : nib<0>(w[u][h][g]);
            a[u][2 + h] = step ? nib<3>(w[u][h][g]) : nib<1>(w[u][h][g]);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int np = 0; np < NP; ++np) {
            const uint2 b = qb[(((nt * NP + np) * NG + g) * 2 + step) * 32];
#pragma unroll
            for (int u = 0; u < 2; ++u) mma_bf16(c[u][nt], a[u][0], a[u][1], a[u][2], a[u][3], b.x, b.y);
          }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float k = half(ks[u][i >> 1][g / 2]);
            s[u][nt][i] = g == 0 ? k * c[u][nt][i] : fmaf(k, c[u][nt][i], s[u][nt][i]);
          }
    }
  }

  // Adds the block's values under the weights p (a bit of dead for each that takes no part).
  template <bool MASKED> __device__ __forceinline__ void values(const uint8_t* blk, const float (&p)[NT][4], uint32_t dead) {
    const int rr = lane >> 2, tq = lane & 3;
    const uint8_t* prm = blk + 16 * DH + 64 * NG;  // scales and zeros
    uint32_t vs[2][NG / 2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NG / 2; ++i) vs[h][i] = reinterpret_cast<const uint32_t*>(prm + 4 * NG * (rr + 8 * h))[i];
    // zeros: by this lane's keys rr and rr + 8 (in fp32 arithmetic), or as operands, by the four keys of its columns
    constexpr bool SIMT = CENTRED || MASKED;
    constexpr int NZ = SIMT ? 2 : 4;
    uint32_t vz[NZ][NG / 2];
#pragma unroll
    for (int h = 0; h < NZ; ++h)
#pragma unroll
      for (int i = 0; i < NG / 2; ++i)
        vz[h][i] = reinterpret_cast<const uint32_t*>(prm + 4 * NG * (SIMT ? rr + 8 * h : 2 * tq + (h & 1) + 4 * (h & 2)))[NG / 2 + i];
    uint32_t pb[NT][NP][NG][2];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float s0 = g & 1 ? hi_f(vs[0][g / 2]) : lo_f(vs[0][g / 2]), s1 = g & 1 ? hi_f(vs[1][g / 2]) : lo_f(vs[1][g / 2]);
      const float z0 = (g & 1 ? hi_f(vz[0][g / 2]) : lo_f(vz[0][g / 2])) + (CENTRED ? OFF : 0.f);
      const float z1 = (g & 1 ? hi_f(vz[1][g / 2]) : lo_f(vz[1][g / 2])) + (CENTRED ? OFF : 0.f);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4] = {p[nt][0] * s0, p[nt][1] * s0, p[nt][2] * s1, p[nt][3] * s1};
        auto out = [&](int i) { return MASKED && (dead >> (4 * nt + i) & 1); };
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (out(i)) x[i] = 0.f;
        if (CENTRED) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!out(i)) corr[nt][g][i & 1] = fmaf(x[i], i < 2 ? z0 : z1, corr[nt][g][i & 1]);
        }
#pragma unroll
        for (int np = 0; np < NP; ++np) {
          const uint32_t u0 = NP > 1 ? split_off(x[0], x[1]) : pack_bf16x2(x[0], x[1]);
          const uint32_t u1 = NP > 1 ? split_off(x[2], x[3]) : pack_bf16x2(x[2], x[3]);
          if (MASKED && !CENTRED) {
            // the zeros' part of the tile's last blocks, where an operand's NaN would reach rows that do not see it
            const float r[4] = {lo_f(u0), hi_f(u0), lo_f(u1), hi_f(u1)};
            float add[2] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!out(i)) add[i & 1] = fmaf(r[i], i < 2 ? z0 : z1, add[i & 1]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) add[c] += __shfl_xor_sync(0xffffffffu, add[c], d);
#pragma unroll
              for (int j = 2 * g; j < 2 * g + 2; ++j) {
                o[nt][j][c] += add[c];
                o[nt][j][2 + c] += add[c];
              }
            }
          }
          pb[nt][np][g][0] = transpose8x8(u0);
          pb[nt][np][g][1] = transpose8x8(u1);
        }
      }
    }
    if (!CENTRED) {
#pragma unroll
      for (int j = 0; j < DH / 16; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_bf16(o[nt][j], minus16[0], minus16[1], minus16[2], minus16[3], pb[nt][0][j / 2][0], pb[nt][0][j / 2][1]);
      if (!SIMT) {
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          const uint32_t sel = j / 2 & 1 ? 0x7632 : 0x5410;
          const uint32_t za = __byte_perm(vz[0][j / 4], vz[1][j / 4], sel), zb = __byte_perm(vz[NZ - 2][j / 4], vz[NZ - 1][j / 4], sel);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][j], za, za, zb, zb, pb[nt][0][j / 2][0], pb[nt][0][j / 2][1]);
        }
      }
    }
#pragma unroll
    for (int half = 0; half < DH / 64; ++half) {  // 64 channels, four fragments
      uint32_t w[4];
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(blk + 8 * DH + 512 * half + 16 * lane);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int j = 4 * half + jj;
        const uint32_t a0 = nib<0>(w[jj]), a1 = nib<1>(w[jj]), a2 = nib<2>(w[jj]), a3 = nib<3>(w[jj]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (!CENTRED) {
            mma_bf16(o[nt][j], a0, a1, a2, a3, pb[nt][0][j / 2][0], pb[nt][0][j / 2][1]);
          } else {
            float c[4] = {};
#pragma unroll
            for (int np = NP - 1; np >= 0; --np) mma_bf16(c, a0, a1, a2, a3, pb[nt][np][j / 2][0], pb[nt][np][j / 2][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][j][i] += c[i];
          }
        }
      }
    }
  }

  // Two blocks of 16 keys from key0 on, 16 AW apart, in shared memory.  MASKED: some row does not see all of them, or one is
  // not there (a key that a row does not see may hold anything, a NaN scale too, and takes no part).
  template <bool MASKED>
  __device__ __forceinline__ void two_blocks(const uint8_t* blk0, const uint8_t* blk1, int key0, uint32_t there, float scale_log2) {
    const int rr = lane >> 2;
    float s[2][NT][4];
    scores(blk0, blk1, s);
    bool up = false;
    uint32_t dead[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[u][nt][i] *= scale_log2;
          if (MASKED && (!(there >> u & 1) || key0 + u * 16 * AW + rr + (i >> 1) * 8 > lim[nt][i & 1])) {
            s[u][nt][i] = -INFINITY;
            dead[u] |= 1u << (4 * nt + i);
          }
          up |= s[u][nt][i] > m[nt][i & 1] + LAZY;
        }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = fmaxf(m[nt][c], fmaxf(fmaxf(s[0][nt][c], s[0][nt][2 + c]), fmaxf(s[1][nt][c], s[1][nt][2 + c])));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          const float f = exp2_fast(m[nt][c] - x);
          m[nt][c] = x;
          l[nt][c] *= f;
          if (CENTRED)
#pragma unroll
            for (int g = 0; g < NG; ++g) corr[nt][g][c] *= f;
#pragma unroll
          for (int j = 0; j < DH / 16; ++j) {
            o[nt][j][c] *= f;
            o[nt][j][2 + c] *= f;
          }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[u][nt][i] = exp2_fast(s[u][nt][i] - m[nt][i & 1]);
          l[nt][i & 1] += s[u][nt][i];
        }
    values<MASKED>(blk0, s[0], dead[0]);
    values<MASKED>(blk1, s[1], dead[1]);
  }

  template <int I> __device__ __forceinline__ uint32_t nib(uint32_t x) const { return nibbles<I, CENTRED>(x, mask, sixteen); }
};

template <int DH> __device__ __forceinline__ void copy_block(uint32_t dst, const uint8_t* src, int lane) {
#pragma unroll
  for (int i = 0; i < (kvq_block_bytes(DH) / 16 + 31) / 32; ++i) {
    const int c = i * 32 + lane;
    if (c < kvq_block_bytes(DH) / 16) cp_async16(dst + c * 16, src + c * 16, 16);
  }
}

// weight of a part of maximum m under the common maximum M (a part without keys: m = LOWEST, sums of zero).  Sums are
// added under weights of zero too: a NaN among them stays one.
__device__ __forceinline__ float part_weight(float m, float M) { return exp2f(m - M); }

template <typename T, int DH, int NT, int NP>
__global__ void __launch_bounds__(AW * 32, NT == 2 ? (NP == 1 ? 3 : 2) : NP == 1 ? 4 : 3) kvq_attention_kernel(const __grid_constant__ KvqAttn p) {
  typedef Attn<T, DH, NT, NP> A;
  constexpr int R = A::R, ROW = A::ROW;
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int TILES = 256;
  __shared__ long long scan[AW];
  __shared__ int tile_len[TILES];
  // the schedule, kept out of the registers of the loop over the keys
  __shared__ struct {
    long long share, rest;       // the CTAs' shares: share quanta, the first `rest` one more
    long long begin, end;        // this CTA's
    long long cur, base, unit;   // where it is; its tile's and its unit's first quantum
    int ti, len, nq, q0, q1, seq, head, r0;
  } sc;
  __shared__ float part_m[AW][R], part_l[AW][R], wts[AW][R], row_m[R], row_l[R];
  __shared__ int is_last;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, rr = lane >> 2, tq = lane & 3;
  const int heads = p.c.n_kv_heads, rows = p.T * p.G;

  // this CTA's share of all quanta: the tiles' quanta and running sums, by one warp where it has a lane for each
  const bool few = p.n_tiles <= 32;
  if (few && w != 0) {
    // (waits for the first warp below)
  } else {
    const int lanes = few ? 32 : AW * 32, per = (p.n_tiles + lanes - 1) / lanes;
    long long mine = 0;
    for (int i = tid * per; i < min(p.n_tiles, (tid + 1) * per); ++i) {
      int len;
      mine += tile_quanta(p, i, R, len);
      if (i < TILES) tile_len[i] = len;
    }
    mine *= heads;
    long long sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += y;
    }
    if (!few) {
      if (lane == 31) scan[w] = sum;
      __syncthreads();
      long long before = 0;
#pragma unroll
      for (int i = 0; i < AW; ++i)
        if (i < w) before += scan[i];
      sum += before;
    }
    long long total = few ? __shfl_sync(0xffffffffu, sum, 31) : 0;
    if (!few) {
#pragma unroll
      for (int i = 0; i < AW; ++i) total += scan[i];
    }
    const long long n = min(static_cast<long long>(gridDim.x), quotient(total + MIN_SHARE - 1, MIN_SHARE));
    const long long share = quotient(total, n), rest = total - share * n;
    const long long cur = share * blockIdx.x + min(static_cast<long long>(blockIdx.x), rest);
    const long long end = blockIdx.x < n ? cur + share + (blockIdx.x < rest) : cur;  // (nothing for the other CTAs)
    if (tid == 0) {
      sc.share = share;
      sc.rest = rest;
      sc.begin = sc.cur = cur;
      sc.end = end;
    }
    if (cur < end && sum - mine <= cur && cur < sum) {
      long long base = sum - mine;
      int i = tid * per;
      for (;; ++i) {
        int len = 0;
        if (i < TILES)
          len = tile_len[i];
        else
          tile_quanta(p, i, R, len);
        const long long q = static_cast<long long>(quanta_of(len)) * heads;
        if (cur < base + q) break;
        base += q;
      }
      sc.ti = i;
      sc.base = base;
    }
  }
  // how many keys a tile sees: kept for the first ones, looked up again for the others
  auto len_of = [&](int i) {
    int len;
    if (i < TILES) return tile_len[i];
    tile_quanta(p, i, R, len);
    return len;
  };
  auto begin_of = [&](long long c) { return sc.share * c + min(c, sc.rest); };
  auto owner_of = [&](long long x) {
    const long long longer = sc.rest * (sc.share + 1);
    return static_cast<int>(x < longer ? quotient(x, sc.share + 1) : sc.rest + quotient(x - longer, sc.share));
  };

  for (;;) {
    __syncthreads();
    if (sc.cur >= sc.end) break;
    __syncthreads();
    if (tid == 0) {  // the next unit, or its part
      sc.len = len_of(sc.ti);
      sc.nq = quanta_of(sc.len);
      sc.head = static_cast<int>(quotient(sc.cur - sc.base, sc.nq));
      sc.unit = sc.base + static_cast<long long>(sc.head) * sc.nq;
      sc.q0 = static_cast<int>(sc.cur - sc.unit);
      sc.q1 = static_cast<int>(min(static_cast<long long>(sc.nq), sc.end - sc.unit));
      sc.seq = sc.ti / p.tiles_per_seq;
      sc.r0 = (sc.ti - sc.seq * p.tiles_per_seq) * R;
    }
    __syncthreads();
    {
    const int len = sc.len, q0 = sc.q0, q1 = sc.q1, seq = sc.seq, head = sc.head, r0 = sc.r0;
    const int blocks = min((len + KVQ_BLOCK - 1) / KVQ_BLOCK, (q1 - UNIT_COST) * AW), per_page = p.c.page_tokens / KVQ_BLOCK;
    const int b0 = max(0, q0 - UNIT_COST) * AW + w, count = blocks > b0 ? (blocks - b0 + AW - 1) / AW : 0;
    uint8_t* ring = smem + w * A::STAGES * A::BLK;
    const uint32_t ring_u = smem_u32(ring);
    uint32_t there = 0;  // bit s: stage s holds a block
    const uint8_t* at = nullptr;  // each lane: one of this warp's next 32 blocks
    auto fetch = [&](int i) {
      if (i < count) {
        if ((i & 31) == 0) {
          at = nullptr;
          if (i + lane < count) {
            const int b = b0 + (i + lane) * AW, slot = b / per_page;
            const int page = p.c.table[seq * p.c.ld_table + slot];
            if (page >= 0 && page < p.c.n_pages)
              at = p.c.pool + ((static_cast<size_t>(page) * heads + head) * per_page + (b - slot * per_page)) * A::BLK;
            else
              set_status(p.status, ST_RANGE);
          }
        }
        const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<u64>(at), i & 31));
        const int stage = i % A::STAGES;
        if (src) copy_block<DH>(ring_u + stage * A::BLK, src, lane);
        there = (there & ~(1u << stage)) | (src ? 1u << stage : 0u);
      }
    };
    auto fetch_two = [&](int i) {
      fetch(i);
      fetch(i + 1);
      cp_async_commit();
    };
    A a;
    {
      float q[NT][8];
      a.load_q(p, seq, r0, head, q);
#pragma unroll
      for (int i = 0; i < A::STAGES - 2; i += 2) fetch_two(i);
      a.start(smem + A::WORK, q);
    }
    __syncthreads();
    const int all = a.seen_by_all(p, r0);
    for (int i = 0; i < count; i += 2) {
      __syncwarp();  // (every lane is done with the stages that are written next)
      fetch_two(i + A::STAGES - 2);
      cp_async_wait<A::STAGES / 2 - 1>();
      __syncwarp();
      const int stage = i % A::STAGES, key0 = (b0 + i * AW) * KVQ_BLOCK;
      const uint32_t ok = i + 1 < count ? there >> stage & 3u : there >> stage & 1u;
      const uint8_t* blk = ring + stage * A::BLK;
      if (ok == 3 && all - key0 >= QUANTUM + KVQ_BLOCK - 1)
        a.template two_blocks<false>(blk, blk + A::BLK, key0, 3, p.scale_log2);
      else if (ok)
        a.template two_blocks<true>(blk, blk + A::BLK, key0, ok, p.scale_log2);
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with its ring: the merge buffer lies over them

    float* buf = reinterpret_cast<float*>(smem) + w * R * ROW;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = nt * 8 + 2 * tq + c;
        float sum = a.l[nt][c], corr[A::NG];
#pragma unroll
        for (int g = 0; g < A::NG; ++g) corr[g] = A::CENTRED ? a.corr[nt][g][c] : 0.f;
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, d);
          if (A::CENTRED)
#pragma unroll
            for (int g = 0; g < A::NG; ++g) corr[g] += __shfl_xor_sync(0xffffffffu, corr[g], d);
        }
        if (rr == 0) {
          part_m[w][row] = a.m[nt][c];
          part_l[w][row] = sum;
        }
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          buf[row * ROW + 16 * j + rr] = a.o[nt][j][c] + corr[j / 2];
          buf[row * ROW + 16 * j + rr + 8] = a.o[nt][j][2 + c] + corr[j / 2];
        }
      }
    }
    __syncthreads();
    if (tid < R) {
      float M = LOWEST, L = 0.f;
#pragma unroll
      for (int i = 0; i < AW; ++i) M = fmaxf(M, part_m[i][tid]);
#pragma unroll
      for (int i = 0; i < AW; ++i) {
        const float x = part_weight(part_m[i][tid], M);
        wts[i][tid] = x;
        L += x * part_l[i][tid];
      }
      row_m[tid] = M;
      row_l[tid] = L;
    }
    __syncthreads();
    const int seq = sc.seq, head = sc.head, r0 = sc.r0;
    const bool whole = sc.q1 - sc.q0 == sc.nq;
    // 2 slots a CTA: the first part of its share, and a later one
    float* slot = p.parts + (2 * static_cast<size_t>(blockIdx.x) + (sc.cur != sc.begin)) * slot_floats(DH);
    const float* sm = reinterpret_cast<const float*>(smem);
    for (int i = tid; i < R * DH; i += AW * 32) {
      const int row = i / DH, ch = i - row * DH, gr = r0 + row;
      if (gr >= rows) break;
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < AW; ++k) x = fmaf(wts[k][row], sm[(k * R + row) * ROW + ch], x);
      if (whole) {
        const int t = gr / p.G;
        static_cast<T*>(p.out)[(static_cast<long long>(seq) * p.T + t) * p.ldo +
                               static_cast<long long>(head * p.G + gr - t * p.G) * DH + ch] =
            from_f<T>(row_l[row] == 0.f ? 0.f : x / row_l[row]);
      } else {
        slot[row * DH + ch] = x;
      }
    }
    if (!whole) {
      if (tid < R) *reinterpret_cast<float2*>(slot + MAX_ROWS * DH + 2 * tid) = make_float2(row_m[tid], row_l[tid]);
      const int c0 = owner_of(sc.unit), c1 = owner_of(sc.unit + sc.nq - 1);  // CTAs of this unit
      __syncthreads();
      if (tid == 0) {
        __threadfence();  // (with the barrier before it: all of the CTA's part)
        is_last = atomicAdd(p.counters + c0, 1) == c1 - c0;
      }
      __syncthreads();
      if (is_last) {
        __threadfence();
        if (tid == 0) p.counters[c0] = 0;
        // parts c0..c1: the first in its CTA's first or later slot, the others in their CTA's first; a warp's row
        // at a time, four channels a lane
        const float* parts = p.parts + 2 * static_cast<size_t>(c0) * slot_floats(DH);
        const int shift = sc.unit != begin_of(c0) ? slot_floats(DH) : 0, np = c1 - c0 + 1;
        float* wt = reinterpret_cast<float*>(smem) + w * (A::WEIGHTS / 4 / AW);
        for (int row = w; row < R && r0 + row < rows; row += AW) {
          constexpr int CH = DH / 32, AHEAD = 8;  // channels a lane; parts whose loads are under way together
          auto part = [&](int c) { return parts + (c ? 2 * static_cast<size_t>(c) * slot_floats(DH) : shift); };
          auto load = [&](int c, float (&v)[CH]) {
            const float* at = part(c) + row * DH + lane * CH;
            if (CH == 4)
              *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(at));
            else
              *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(at));
          };
          float v[AHEAD][CH];
#pragma unroll
          for (int i = 0; i < AHEAD; ++i)
            if (i < np) load(i, v[i]);
          float M = LOWEST, L = 0.f;
          for (int c = lane; c < np; c += 32) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(c) + MAX_ROWS * DH + 2 * row));
            wt[c] = ml.x;
            wt[c + KVQ_MAX_CTAS] = ml.y;
            M = fmaxf(M, ml.x);
          }
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
          for (int c = lane; c < np; c += 32) {
            const float x = part_weight(wt[c], M);
            L = fmaf(x, wt[c + KVQ_MAX_CTAS], L);
            wt[c] = x;
          }
          L = warp_sum(L);
          __syncwarp();
          float x[CH] = {};
          for (int c0 = 0; c0 < np; c0 += AHEAD) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
              if (c0 + i < np) {
                const float f = wt[c0 + i];
#pragma unroll
                for (int k = 0; k < CH; ++k) x[k] = fmaf(f, v[i][k], x[k]);
                if (c0 + AHEAD + i < np) load(c0 + AHEAD + i, v[i]);
              }
            }
          }
          __syncwarp();
          const int gr = r0 + row, t = gr / p.G;
          T* dst = static_cast<T*>(p.out) + (static_cast<long long>(seq) * p.T + t) * p.ldo +
                   static_cast<long long>(head * p.G + gr - t * p.G) * DH + lane * CH;
#pragma unroll
          for (int i = 0; i < CH; ++i) dst[i] = from_f<T>(L == 0.f ? 0.f : x[i] / L);
        }
      }
    }
    __syncthreads();  // the merge buffer becomes rings again
    if (tid == 0) {
      sc.cur = sc.unit + sc.q1;
      if (sc.cur == sc.base + static_cast<long long>(sc.nq) * heads) {
        sc.base = sc.cur;
        ++sc.ti;
      }
    }
  }
}

template <typename T, int DH, int NT, int NP>
cudaError_t launch(KvqAttn p, cudaStream_t s) {
  typedef Attn<T, DH, NT, NP> A;
  p.tiles_per_seq = (p.T * p.G + A::R - 1) / A::R;
  p.n_tiles = p.c.n_seqs * p.tiles_per_seq;
  static DeviceOnce configured;
  cudaError_t e = max_dynamic_smem_once(reinterpret_cast<const void*>(kvq_attention_kernel<T, DH, NT, NP>), A::SMEM, configured);
  if (e != cudaSuccess) return e;
  // as many CTAs as fit at once, per device
  static std::atomic<int> fits[64];
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < 64;
  int grid = cached ? fits[dev].load(std::memory_order_relaxed) : 0;
  if (grid == 0) {
    int sms = 0, per_sm = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kvq_attention_kernel<T, DH, NT, NP>, AW * 32, A::SMEM)) != cudaSuccess)
      return e;
    grid = std::min(KVQ_MAX_CTAS, std::max(1, per_sm) * sms);
    if (cached) fits[dev].store(grid, std::memory_order_relaxed);
  }
  return launch_chain(kvq_attention_kernel<T, DH, NT, NP>, dim3(grid), dim3(AW * 32), A::SMEM, s, p);
}

}  // namespace

size_t kvq_scratch_bytes() {
  return KVQ_MAX_CTAS * sizeof(int) + 2 * static_cast<size_t>(KVQ_MAX_CTAS) * slot_floats(128) * sizeof(float);
}

cudaError_t launch_kvq_attention(const KvqView& c, int head_dim, const void* q, long long ldq, const int32_t* q_pos, int T,
                                 int n_heads, float scale, cb_dtype dt, void* out, long long ldo, void* scratch,
                                 int32_t* status, cudaStream_t s) {
  KvqAttn p = {};
  p.c = c;
  p.q = q;
  p.ldq = ldq;
  p.q_pos = q_pos;
  p.T = T;
  p.G = n_heads / c.n_kv_heads;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  p.ldo = ldo;
  p.counters = static_cast<int*>(scratch);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + KVQ_MAX_CTAS * sizeof(int));
  p.status = status;
  const bool two = T * p.G > 8;
  if (dt == CB_BF16) {
    if (head_dim == 128) return two ? launch<bf16, 128, 2, 1>(p, s) : launch<bf16, 128, 1, 1>(p, s);
    return two ? launch<bf16, 64, 2, 1>(p, s) : launch<bf16, 64, 1, 1>(p, s);
  }
  if (head_dim == 128) return two ? launch<float, 128, 2, 3>(p, s) : launch<float, 128, 1, 3>(p, s);
  return two ? launch<float, 64, 2, 3>(p, s) : launch<float, 64, 1, 3>(p, s);
}

}  // namespace cb
